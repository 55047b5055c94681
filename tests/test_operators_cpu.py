"""Rotary, paged-cache and score-modified operators without a GPU: refusals of the C ABI and of the
Python entry points, the page arithmetic, the tables, and the tests' own 64-bit forms."""
import ctypes
import importlib.util
import math
import re
import shutil
import subprocess
from pathlib import Path

import numpy as np
import pytest
import torch

import exact_attention_107_b200 as fa
import operator_refs as ref

CSRC = Path(fa.__file__).resolve().parent / "csrc"
P = ctypes.c_void_p(0x10000)        # an aligned, never-dereferenced fake address
U = ctypes.c_void_p(0x10008)        # 8-byte aligned only
O = ctypes.c_void_p(0x10002)        # not even 4
Z = None


def strides(*s):
    return (ctypes.c_longlong * 3)(*s)


S = strides(1024, 64, 64)


# ----------------------------------------------------------------------------- C ABI refusals
def _fwd_mod(q=P, k=P, v=P, o=P, lse=P, plan=Z, slopes=Z, cap=0.0, B=1, H=2, Hkv=1, N=256, D=64, scale=0.125, causal=0,
             dtype=0):
    return fa.load_library().fa_fwd_mod(q, k, v, o, lse, plan, slopes, cap, B, H, Hkv, N, D, scale, causal, dtype, None)


def _bwd_mod(dk=P, ws=P, n=1 << 30, plan=Z, slopes=Z, cap=0.0, B=1, H=2, Hkv=1, N=256, D=64, scale=0.125, causal=0,
             dtype=0):
    return fa.load_library().fa_bwd_mod(P, P, P, P, P, P, P, dk, P, ws, n, plan, slopes, cap, B, H, Hkv, N, D, scale,
                                        causal, dtype, None)


COMMON = [
    (dict(H=3, Hkv=2), 2), (dict(Hkv=0), 2), (dict(B=0), 2), (dict(N=0), 2), (dict(D=256), 3), (dict(D=80), 3),
    (dict(cap=-1.0), 10), (dict(cap=float("inf")), 10), (dict(cap=float("nan")), 10), (dict(scale=0.0), 10),
    (dict(scale=float("inf")), 10), (dict(causal=2), 10), (dict(plan=P, causal=1), 10), (dict(dtype=2), 10),
    (dict(plan=U), 4), (dict(slopes=O), 4), (dict(plan=P, N=300000), 2),
]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(q=Z), 1), (dict(lse=Z), 1), (dict(o=U), 4)])
def test_fwd_mod_refusals(kw, code):
    assert _fwd_mod(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [(dict(dk=Z), 1), (dict(dk=U), 4), (dict(n=100), 8), (dict(ws=Z), 8)])
def test_bwd_mod_refusals(kw, code):
    assert _bwd_mod(**kw) == code


@pytest.mark.parametrize("args,code", [
    ((Z, 1 << 20, Z, Z, 1, 100, 1, 0), 8), ((P, 10, Z, Z, 1, 100, 1, 0), 8), ((P, 1 << 20, Z, Z, 0, 100, 1, 0), 2),
    ((P, 1 << 20, Z, Z, 1, 300000, 1, 0), 2), ((P, 1 << 20, Z, Z, 1, 100, 2, 0), 10),
    ((P, 1 << 20, Z, Z, 1, 100, 1, -1), 10), ((P, 1 << 20, Z, P, 1, 100, 0, 0), 10), ((P, 1 << 20, P, P, 1, 100, 1, 0), 10),
    ((P, 1 << 20, Z, P, 1, 100, 1, 5), 10), ((U, 1 << 20, Z, Z, 1, 100, 1, 0), 4), ((P, 1 << 20, O, Z, 1, 100, 1, 0), 4),
])
def test_mask_plan_refusals(args, code):
    assert fa.load_library().fa_mask_plan(*args, None) == code


def test_mask_plan_size():
    # per 128 rows: 128 intervals, 2 tile ranges and an entry of two orders, of 8 bytes each
    assert fa.fa_mask_plan_size(1, 1) == 8 * (128 + 2 + 1)
    assert fa.fa_mask_plan_size(3, 129) == 3 * 2 * 8 * (128 + 2 + 1)
    assert fa.fa_mask_plan_size(1, 262144) > 0 and fa.fa_mask_plan_size(1, 262145) == 0
    assert fa.fa_mask_plan_size(0, 5) == 0


def _rotary(q=P, k=P, qo=P, ko=P, table=P, pos=Z, qs=S, ks=S, ps=0, rows=100, B=1, H=2, Hkv=1, N=10, D=64, R=64, il=0,
            inv=0, dtype=0):
    return fa.load_library().fa_rotary(q, k, qo, ko, table, pos, qs, ks, ps, rows, B, H, Hkv, N, D, R, il, inv, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=Z), 1), (dict(ko=Z), 1), (dict(table=Z), 1), (dict(qs=Z), 1), (dict(H=0, Hkv=0), 2), (dict(H=-1), 2),
    (dict(N=0), 2), (dict(B=1 << 20, N=1 << 20), 2), (dict(D=48), 3), (dict(R=0), 10), (dict(R=3), 10), (dict(R=66), 10),
    (dict(rows=0), 10), (dict(q=U), 4), (dict(pos=O), 4), (dict(qs=strides(1024, 60, 64)), 4),
    (dict(ks=strides(-8, 64, 64)), 4), (dict(il=2), 10), (dict(inv=-1), 10), (dict(dtype=7), 10), (dict(ps=-1), 10),
])
def test_rotary_refusals(kw, code):
    assert _rotary(**kw) == code


def _append(k=P, v=P, kp=P, vp=P, q=P, qo=P, bt=P, sl=P, nl=Z, table=P, ks=S, vs=S, qs=S, rows=100, width=4, pages=10,
            page=16, B=1, H=2, Hkv=1, T=3, D=64, R=64, il=0, dtype=0):
    return fa.load_library().fa_paged_append(k, v, kp, vp, q, qo, bt, sl, nl, table, ks, vs, qs, rows, width, pages, page,
                                             B, H, Hkv, T, D, R, il, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=Z), 1), (dict(vp=Z), 1), (dict(bt=Z), 1), (dict(q=Z), 1), (dict(vs=Z), 1), (dict(Hkv=0), 2), (dict(T=0), 2),
    (dict(page=4), 2), (dict(page=24), 2), (dict(page=512), 2), (dict(width=0), 2), (dict(pages=0), 2),
    (dict(width=1 << 28), 2), (dict(D=40), 3), (dict(table=Z), 10), (dict(R=65), 10), (dict(R=0), 10), (dict(kp=U), 4),
    (dict(sl=O), 4), (dict(nl=O), 4), (dict(vs=strides(4, 64, 64)), 4), (dict(il=3), 10), (dict(dtype=-1), 10),
])
def test_append_refusals(kw, code):
    assert _append(**kw) == code


def _decode(q=P, kp=P, bt=P, sl=P, o=P, lse=P, ws=P, n=1 << 30, slopes=Z, cap=0.0, window=0, width=4, pages=10, page=16,
            B=1, H=2, Hkv=1, T=1, D=64, scale=0.125, dtype=0):
    return fa.load_library().fa_paged_attention(q, kp, P, bt, sl, o, lse, ws, n, slopes, cap, window, width, pages, page,
                                                B, H, Hkv, T, D, scale, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=Z), 1), (dict(lse=Z), 1), (dict(T=0), 2), (dict(T=65), 2), (dict(H=3, Hkv=2), 2), (dict(B=5000), 2),
    (dict(page=12), 2), (dict(width=0), 2), (dict(pages=1 << 30), 2), (dict(D=100), 3), (dict(q=U), 4), (dict(bt=O), 4),
    (dict(scale=-1.0), 10), (dict(cap=float("nan")), 10), (dict(window=-1), 10), (dict(dtype=3), 10), (dict(ws=Z), 8),
    (dict(n=0), 8), (dict(ws=U), 4),
])
def test_paged_attention_refusals(kw, code):
    assert _decode(**kw) == code


def test_status_string_of_bad_indexes():
    assert fa.status_string(13).startswith("FA_ERR_INDEX")


# ----------------------------------------------------------------------------- Python refusals
def test_python_entry_points_refuse_cpu_tensors_and_types():
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.attention_forward(q, q, q, softcap=30.0)
    with pytest.raises(ValueError, match="CUDA"):
        fa.rotary_forward(q, q, fa.rotary_table(4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        fa.paged_append(q, q, q, q, i[None], i)
    with pytest.raises(ValueError, match="CUDA"):
        fa.paged_attention(q, q, q, i[None], i)
    with pytest.raises(ValueError):
        fa.attention_mask(1, 4, device="cpu")
    with pytest.raises(ValueError):
        fa.rotary_forward(None, None, fa.rotary_table(4, 64))
    with pytest.raises(ValueError, match="needs a table"):
        fa.paged_append(q, q, q, q, i[None], i, q=q)
    with pytest.raises(ValueError, match="deterministic"):
        fa.attention_backward(q, q, q, q, None, q, softcap=1.0, deterministic=True)


# ----------------------------------------------------------------------------- page arithmetic
HOST = """
#include "paged_index.h"
extern "C" int host_page_of(const int* row, int width, int shift, int pages, long long p) {
  return fa::page_of(row, width, shift, pages, p);
}
extern "C" long long host_row(int page, int heads, int hk, long long p, int shift) {
  return fa::page_row_of(page, heads, hk, p, shift);
}
extern "C" int host_append(int len, int fresh, int T, int n, const int* row, int width, int shift, int pages,
                           long long* position, int* page) {
  const fa::AppendSlot s = fa::append_slot(len, fresh, T, n, row, width, shift, pages);
  *position = s.position;
  *page = s.page;
  return s.real;
}
extern "C" int host_first(int p, int window) { return fa::first_seen(p, window); }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("paged")
    (d / "host.cc").write_text(HOST)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", str(CSRC), str(d / "host.cc"), "-o",
                    str(d / "host.so")], check=True)
    lib = ctypes.CDLL(str(d / "host.so"))
    lib.host_page_of.argtypes = [ctypes.c_void_p] + [ctypes.c_int] * 3 + [ctypes.c_longlong]
    lib.host_row.argtypes = [ctypes.c_int] * 3 + [ctypes.c_longlong, ctypes.c_int]
    lib.host_row.restype = ctypes.c_longlong
    lib.host_append.argtypes = [ctypes.c_int] * 4 + [ctypes.c_void_p] + [ctypes.c_int] * 3 + [ctypes.c_void_p] * 2
    return lib


def test_bad_pages_are_never_followed(host):
    row = (ctypes.c_int * 4)(2, 9, -1, 10)
    for p in list(range(-3, 70)) + [2 ** 31 - 1, 2 ** 40, -2 ** 40]:
        want = -1
        if 0 <= p < 64 and 0 <= row[p // 16] < 10:
            want = row[p // 16]
        assert host.host_page_of(row, 4, 4, 10, p) == want
    pos, page = ctypes.c_longlong(), ctypes.c_int()
    for length in (0, 1, 16, 17, 64, 65, 2 ** 31 - 1, -5):
        for fresh in (-1, 0, 1, 3, 4, 2 ** 31 - 1):
            for n in range(3):
                real = host.host_append(length, fresh, 3, n, row, 4, 4, 10, ctypes.byref(pos), ctypes.byref(page))
                p = length - fresh + n
                assert bool(real) == (n < fresh) and pos.value == p
                ok = n < fresh <= 3 and 0 <= p < 64 and 0 <= row[p // 16] < 10
                assert page.value == (row[p // 16] if ok else -1)


def test_rows_pass_32_bits(host):
    assert host.host_row(2 ** 31 - 1, 64, 63, 255, 8) == ((2 ** 31 - 1) * 64 + 63) * 256 + 255
    assert host.host_first(10, 0) == 0 and host.host_first(10, 11) == 0 and host.host_first(10, 10) == 1
    assert host.host_first(10, 1) == 10 and host.host_first(-4, 3) == 0
    assert host.host_first(2 ** 31 - 2, 2 ** 31 - 1) == 0


# ----------------------------------------------------------------------------- tables
def test_rotary_table():
    t = fa.rotary_table(5000, 64, 10000.0)
    assert t.shape == (5000, 64) and t.dtype == torch.float32
    for p, i in ((0, 0), (1, 0), (4999, 0), (4999, 31), (777, 13)):
        angle = p * 10000.0 ** (-2 * i / 64)
        assert abs(float(t[p, i]) - math.cos(angle)) <= 2.0 ** -24 and abs(float(t[p, 32 + i]) - math.sin(angle)) <= 2.0 ** -24
    linear = fa.rotary_table(400, 64, scaling="linear", factor=4.0)
    assert (linear[::4] - fa.rotary_table(100, 64)).abs().max() <= 2.0 ** -24
    wide = fa.rotary_table(400, 64, scaling="base", factor=4.0)
    plain = fa.rotary_table(400, 64)
    assert torch.equal(wide[:, 0], plain[:, 0]) and (wide[4 * 90, 31] - plain[90, 31]).abs() <= 2.0 ** -23
    parts = fa.rotary_table(400, 64, scaling="by_parts", factor=4.0, original_length=100, low=1.0, high=8.0)
    size = 0.1 * math.log(4.0) + 1.0
    assert abs(float(parts[1, 0]) - size * math.cos(1.0)) <= 2.0 ** -23                      # 16 turns: kept
    assert abs(float(parts[300, 63]) - size * math.sin(75 * 10000.0 ** (-62 / 64))) <= 2.0 ** -23   # under one: stretched
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(factor=0.5), dict(scaling="other"),
                dict(scaling="by_parts"), dict(scaling="base", rotary_dim=2), dict(length=0)):
        with pytest.raises(ValueError):
            fa.rotary_table(**{**dict(length=4, rotary_dim=8), **bad})


# ----------------------------------------------------------------------------- the capped scores' polynomial
def test_tanh_polynomial_is_the_fit_and_keeps_its_bound():
    spec = importlib.util.spec_from_file_location("gen_tanh_poly", CSRC / "gen_tanh_poly.py")
    g = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(g)
    text = (CSRC / "sm100_ptx.cuh").read_text()
    words = re.findall(r"kTanhC\d = -?[0-9.]+f;\s*// 0x([0-9a-f]{8})", text)
    values = re.findall(r"kTanhC\d = (-?[0-9.]+)f;", text)
    c = np.array([np.frombuffer(bytes.fromhex(w)[::-1], np.float32)[0] for w in words])
    assert len(c) == g.TERMS and np.array_equal(c, g.remez_relative().astype(np.float32))
    assert np.array_equal(c, np.array([float(v) for v in values]).astype(np.float32))
    assert f"kTanhPolyLimit = {g.LIMIT}f" in text
    z = np.linspace(1e-7, g.LIMIT, 300001).astype(np.float32)
    # 5.65e-7 of the fit and a rounding of 2^-24 at each of the last steps
    assert np.abs(g.eval_f32(z, c).astype(np.float64) / np.tanh(z.astype(np.float64)) - 1).max() <= 5.7e-7 + 4 * 2.0 ** -24


# ----------------------------------------------------------------------------- the 64-bit forms
@pytest.mark.parametrize("cap,alibi,kind", [(0.0, False, "documents"), (3.0, True, "documents"), (2.0, False, "window"),
                                            (0.0, True, "prefix")])
def test_reference_gradients_against_differences(cap, alibi, kind):
    """The formulas that the GPU's gradients are held to, against central differences in 64 bits."""
    B, H, Hkv, N, D = 2, 4, 2, 7, 3
    g = torch.Generator().manual_seed(1)
    r = lambda h: torch.randn(B, h, N, D, generator=g, dtype=torch.float64)
    x = {"q": r(H), "k": r(Hkv), "v": r(Hkv)}
    do = r(H)
    seen = {"documents": ref.visible(B, N, documents=torch.tensor([[0, 0, 1, 1, 1, -1, -1], [2, 2, 2, 2, -1, 2, 2]])),
            "window": ref.visible(B, N, causal=False, window=2),
            "prefix": ref.visible(B, N, prefix=torch.tensor([3, 0]))}[kind]
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.7]) if alibi else None
    val, bound = ref.attention(x["q"], x["k"], x["v"], do, 0.6, seen, cap, slopes)
    assert all((bound[n] >= 0).all() for n in bound)

    def loss():
        return (ref.attention(x["q"], x["k"], x["v"], None, 0.6, seen, cap, slopes)[0]["O"] * do).sum()

    h = 1e-5
    for name, grad in (("q", "dQ"), ("k", "dK"), ("v", "dV")):
        flat = x[name].view(-1)
        for i in range(0, flat.numel(), 5):
            was = flat[i].item()
            flat[i] = was + h
            up = loss()
            flat[i] = was - h
            down = loss()
            flat[i] = was
            assert abs((up - down) / (2 * h) - val[grad].reshape(-1)[i]) < 1e-8


def test_reference_turn_is_its_own_transpose():
    g = torch.Generator().manual_seed(2)
    a, b = (torch.randn(2, 3, 5, 8, generator=g, dtype=torch.float64) for _ in range(2))
    table, pos = fa.rotary_table(9, 6, 10.0, scaling="by_parts", factor=2.0, original_length=4), torch.randint(0, 9, (2, 5), generator=g)
    for il in (False, True):
        ya = ref.turn(a, table, pos, il)[0]
        zb = ref.turn(b, table, pos, il, True)[0]
        assert abs((ya * b).sum() - (a * zb).sum()) < 1e-12
