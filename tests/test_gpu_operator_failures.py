"""The rotary, paged-cache and score-modified kernels' bounded waits and device-side checks.

Child processes load the library's test builds: libfa_timeout_test.so, whose pipeline waits last 100
clocks, so that each kernel runs one out, takes its error path and reports FA_ERR_TIMEOUT with the
context left usable; and libfa_debug.so, whose checks of indices and of warp convergence must stay
silent while the results match the normal build's."""
import json
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

ROOT = Path(__file__).resolve().parents[1]

CHILD = r"""
import json, sys
import torch
sys.path.insert(0, sys.argv[1])
import exact_attention_107_b200 as fa
import exact_attention_107_b200._binding as b
normal = b.LIB_PATH

def use(path):
    b.LIB_PATH, b._lib = path, None

def rand(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()

def modified(D, H, Hkv, N, cap, alibi, kind, dtype):
    q, k, v, do = (rand(2, h, N, D, seed=i, dtype=dtype) for i, h in enumerate((H, Hkv, Hkv, H)))
    slopes = torch.tensor([0.5 / (h + 1) for h in range(H)]).cuda() if alibi else None
    ids = (torch.arange(N) * 5 // N).int().repeat(2, 1)
    ids[1, N // 2:] = -1
    mask = fa.attention_mask(2, N, documents=ids.cuda(), causal=kind == "causal") if kind else None
    more = dict(mask=mask, softcap=cap, alibi_slopes=slopes)
    o, lse = fa.attention_forward(q, k, v, causal=mask is None, **more)
    st = [fa.fa_device_status(True)]
    dq, dk, dv = fa.attention_backward(q, k, v, o, lse, do, causal=mask is None, **more)
    return st + [fa.fa_device_status(True)], (o, lse, dk, dv)

def paged(D, H, Hkv, T, lens, page, cap, window, dtype):
    q = rand(len(lens), H, T, D, dtype=dtype)
    wide = -(-max(lens) // page)
    kp, vp = (rand(len(lens) * wide, Hkv, page, D, seed=s, dtype=dtype) for s in (1, 2))
    bt = torch.arange(len(lens) * wide, dtype=torch.int32).view(len(lens), wide).cuda()
    out = fa.paged_attention(q, kp, vp, bt, torch.tensor(lens, dtype=torch.int32).cuda(), softcap=cap, window=window)
    return [fa.fa_device_status(True)], out

def turned(D, R, interleaved):
    q, k = rand(2, 3, 5, D), rand(2, 1, 5, D, seed=1)
    out = fa.rotary_forward(q, k, fa.rotary_table(5, R).cuda(), interleaved=interleaved)
    return [fa.fa_device_status(True)], out

bf, hf = torch.bfloat16, torch.float16
cases = {
    "mod_64": lambda: modified(64, 4, 2, 600, 0.0, False, "causal", bf),
    "mod_128_cap": lambda: modified(128, 2, 1, 600, 20.0, False, "full", hf),
    "mod_128_bias": lambda: modified(128, 3, 1, 500, 0.0, True, "full", bf),
    "mod_64_both": lambda: modified(64, 2, 2, 500, 1.0, True, None, bf),
    "paged_128": lambda: paged(128, 8, 2, 1, [5000, 300, 0], 16, 0.0, 0, bf),
    "paged_256": lambda: paged(256, 8, 8, 3, [3000, 2900], 32, 30.0, 700, hf),
    "paged_64": lambda: paged(64, 40, 4, 4, [900, 4000], 8, 0.0, 0, bf),
}
out = {}
if sys.argv[2] == "timeout":
    use(normal.with_name("libfa_timeout_test.so"))
    for name, f in cases.items():
        out[name] = f()[0]
    torch.cuda.synchronize()
else:
    cases.update(turned=lambda: turned(96, 50, False), turned_il=lambda: turned(128, 64, True))
    want = {name: f()[1] for name, f in cases.items()}
    use(normal.with_name("libfa_debug.so"))
    for name, f in cases.items():
        st, got = f()
        out[name] = st + [int(not all(torch.equal(x, y) for x, y in zip(got, want[name])))]
print(json.dumps(out))
"""


def run(kind):
    r = subprocess.run([sys.executable, "-c", CHILD, str(ROOT), kind], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_waits_that_run_out_end_with_a_status(cuda_ok):
    out = run("timeout")
    for name, codes in out.items():
        assert all(c == 7 for c in codes), (name, codes)


def test_debug_build_is_silent_and_agrees(cuda_ok):
    out = run("debug")
    for name, codes in out.items():
        assert not any(codes), (name, codes)
