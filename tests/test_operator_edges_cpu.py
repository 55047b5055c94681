"""Edges of the rotary, paged-cache and score-modified operators without a GPU: index arithmetic at
the ends of its range, arguments beyond C's types, and the package without one of its parts."""
import ctypes
import importlib.util
import re
import shutil
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest

import exact_attention_107_b200 as fa
from exact_attention_107_b200 import build

ROOT = Path(__file__).resolve().parents[1]
CSRC = Path(fa.__file__).resolve().parent / "csrc"

HOST = """
#include "paged_index.h"
extern "C" void host_span(int len, int positions, int T, int window, int tile, int* out) {
  const fa::Span s = fa::span_of(len, positions, T, window, tile);
  out[0] = s.len, out[1] = s.first, out[2] = s.tile0, out[3] = s.ntiles;
}
"""


def test_tiles_of_the_longest_caches(tmp_path):
    """A decode step's span, by the host compiler with signed overflow trapped: lengths up to the
    largest that a table may have, 2^31 - 8."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "host.cc").write_text(HOST)
    subprocess.run([cxx, "-std=c++17", "-O1", "-ftrapv", "-shared", "-fPIC", "-I", str(CSRC), str(tmp_path / "host.cc"),
                    "-o", str(tmp_path / "host.so")], check=True)
    lib = ctypes.CDLL(str(tmp_path / "host.so"))
    out = (ctypes.c_int * 4)()
    most = 2 ** 31 - 8
    for length in (-2 ** 31, -1, 0, 1, 127, 128, 129, 5000, most - 128, most - 1, most, 2 ** 31 - 1):
        for positions in (8, 4096, most):
            for T in (1, 5, 64):
                for window in (0, 1, 128, 1000, 2 ** 31 - 1):
                    lib.host_span(length, positions, T, window, 128, out)
                    n = min(max(length, 0), positions)
                    p = n - T                                   # the first row's position
                    first = p - window + 1 if window and p >= window else 0
                    tiles = -(-n // 128) - first // 128 if n else 0
                    assert tuple(out) == (n, first, first // 128, tiles)
                    assert (first // 128 + tiles) * 128 - 1 <= 2 ** 31 - 1   # the last tile's last position is an int


@pytest.mark.parametrize("beyond", [2 ** 31, 2 ** 32 + 1, 2 ** 64 + 1, -2 ** 31 - 1, -2 ** 32 + 1, -10 ** 30])
def test_integers_beyond_c_are_not_cut(beyond):
    """ctypes would pass a size of 2^32 + 1 as 1."""
    P = ctypes.c_void_p(0x10000)                                # never followed: the call is refused before
    lib = fa.load_library()
    assert fa.fa_mask_plan_size(1, beyond) == 0
    assert fa.fa_paged_workspace_size(beyond, 1, 1, 1, 64) == 0 and fa.fa_paged_workspace_size(1, 1, 1, beyond, 64) == 0
    assert lib.fa_mask_plan(P, 1 << 20, None, None, 1, beyond, 1, 0, None) == 2
    assert lib.fa_mask_plan(P, 1 << 20, None, None, beyond, 4, 1, 0, None) in (2, 8)
    s = (ctypes.c_longlong * 3)(64, 64, 64)
    append = lambda T, rows: lib.fa_paged_append(P, P, P, P, None, None, P, P, None, P, s, s, None, rows, 1, 1, 16, 2, 0, 1, T,
                                                 64, 64, 0, 0, None)
    assert append(beyond, 10) == 2
    if beyond < 0:
        assert lib.fa_mask_plan(P, 1 << 20, None, None, 1, 4, 1, beyond, None) == 10
        assert append(1, beyond) == 10


@pytest.mark.parametrize("cap", [1e-50, -1e-50, 1e-45, 1e-40, 2.4e38, 3e38, 1e39, float("inf"), float("nan"), -1.0])
def test_caps_without_finite_factors_are_refused(cap):
    """softcap log2(e) and scale / softcap as floats; a cap that is 0 only as a float is not "none"."""
    P = ctypes.c_void_p(0x10000)
    lib = fa.load_library()
    assert lib.fa_fwd_mod(P, P, P, P, P, None, None, cap, 1, 2, 1, 256, 64, 0.125, 0, 0, None) == 10
    assert lib.fa_bwd_mod(P, P, P, P, P, P, P, P, P, P, 1 << 30, None, None, cap, 1, 2, 1, 256, 64, 0.125, 0, 0, None) == 10
    assert lib.fa_paged_attention(P, P, P, P, P, P, P, P, 1 << 30, None, cap, 0, 4, 10, 16, 1, 2, 1, 1, 64, 0.125, 0, None) == 10


def python(code):
    r = subprocess.run([sys.executable, "-W", "always", "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r


def test_the_library_serves_without_the_module_of_the_small_calls():
    """_fast.so belongs to one build of torch; without it everything goes through the Python path."""
    r = python("""
import sys
sys.modules["exact_attention_107_b200._fast"] = None       # importing it raises ImportError
import torch
import exact_attention_107_b200 as fa
from exact_attention_107_b200 import build
import exact_attention_107_b200._binding as base
assert fa.fa_version() > 0 and base._fast is None and not base.fast_path(None)
q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
for call in (lambda: fa.rotary_forward(q, q, fa.rotary_table(4, 64)), lambda: fa.attention_forward(q, q, q, softcap=1.0)):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise SystemExit("not refused")
""")
    assert "_fast.so is missing" in r.stderr


def test_another_torch_rebuilds_the_module_of_the_small_calls(tmp_path, monkeypatch):
    """Nothing but _fast.so depends on torch: a new one makes build() compile that, and only that."""
    calls = []
    monkeypatch.setattr(build, "up_to_date", lambda: True)
    monkeypatch.setattr(build, "FAST_STAMP", tmp_path / "_build" / "fast.stamp")
    monkeypatch.setattr(build, "FAST_MODULE", tmp_path / "_fast.so")
    monkeypatch.setattr(build, "_compile", lambda *a: calls.append("cuda"))

    def run(cmd, **kw):
        calls.append("fast")
        Path(cmd[cmd.index("-o") + 1]).write_text("")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    build.build()
    assert calls == ["fast"] and (tmp_path / "_fast.so").exists()
    build.build()
    assert calls == ["fast"]
    monkeypatch.setattr(build, "fast_stamp", lambda: "torch 99 cpython-399")
    build.build()
    build.build()
    assert calls == ["fast", "fast"]


def test_import_under_a_torch_without_cuda():
    """Which lacks the CUDA bindings: importing works, a call is refused for its tensors."""
    python("""
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    delattr(torch._C, name)
import exact_attention_107_b200 as fa
assert fa.rotary_table(4, 8).shape == (4, 8)
q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
try:
    fa.attention_forward(q, q, q, softcap=1.0)
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise SystemExit("not refused")
""")


def test_inverse_of_the_tanh_polynomial():
    """The header's chord is the generator's, and the steps from it leave 2^-22."""
    spec = importlib.util.spec_from_file_location("gen_tanh_poly", CSRC / "gen_tanh_poly.py")
    g = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(g)
    c = g.remez_relative().astype(np.float32)
    text = (CSRC / "sm100_ptx.cuh").read_text()
    for name, want in zip(("kTanhAtLimit", "kTanhChord"), g.chord(c)):
        value, word = re.search(rf"{name} = ([0-9.]+)f;\s*// 0x([0-9a-f]{{8}})", text).groups()
        assert np.float32(value) == want and np.frombuffer(bytes.fromhex(word)[::-1], np.float32)[0] == want
    t = np.linspace(float(g.chord(c)[0]), 1.0, 300001).astype(np.float32)
    z = g.inverse_f32(t, c).astype(np.float64)
    p = z * np.polynomial.polynomial.polyval(z * z, c.astype(np.float64))
    assert np.abs(p - t).max() <= 2.0 ** -22 and (np.diff(z) >= -2.0 ** -21).all() and z[0] >= g.LIMIT - 2.0 ** -21
