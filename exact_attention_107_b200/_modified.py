"""Score-modified attention: shared key-value heads, interval masks, capped scores and a distance
bias (argument marshalling for fa_mask_plan, fa_fwd_mod and fa_bwd_mod)."""
from __future__ import annotations

import contextlib

import torch
from torch.autograd.function import once_differentiable

from . import _binding as base

DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1}


@contextlib.contextmanager
def launch_on(device, stream):
    """Makes `device` and `stream` (None: the device's current stream; a torch.cuda.Stream or a raw
    cudaStream_t) current, so that what a call allocates belongs to the stream its kernels run on.
    Yields a function that registers an output for use on the caller's own stream too."""
    caller = torch.cuda.current_stream(device)
    if stream is None:
        if torch.cuda.current_device() == device.index:
            yield lambda t: t
        else:
            with torch.cuda.device(device):
                yield lambda t: t
        return
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")

    def keep(t):
        if t is not None and stream != caller:
            t.record_stream(caller)
        return t

    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield keep


def check_on(t, name, dtype, shape, device) -> None:
    base._check(t, name, dtype, shape)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def dtype_code(t, name) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in DTYPE_CODES:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float16, got {t.dtype}")
    return DTYPE_CODES[t.dtype]


# ----------------------------------------------------------------------------- masks
class AttentionMask:
    """Which keys each row may see, for B batch elements of N rows: the plan of fa_mask_plan on
    its device.  Made by attention_mask; any number of calls may use it."""

    def __init__(self, plan: torch.Tensor, B: int, N: int):
        self.plan, self.B, self.N = plan, B, N


def fa_mask_plan_size(B: int, N: int) -> int:
    return int(base.load_library().fa_mask_plan_size(B, N))


def fa_mask_plan(plan, documents, prefix, B: int, N: int, causal: bool, window: int, stream=None) -> None:
    """Fills `plan` (a CUDA tensor of at least fa_mask_plan_size bytes) from int32 document ids
    (B,N) or None, and int32 prefix lengths (B) or None."""
    pp, pn = base._ws(plan)
    if documents is not None:
        check_on(documents, "documents", torch.int32, (B, N), plan.device)
    if prefix is not None:
        check_on(prefix, "prefix", torch.int32, (B,), plan.device)
    with launch_on(plan.device, stream):
        base._raise(base.load_library().fa_mask_plan(pp, pn, base._p(documents), base._p(prefix), B, N, int(causal),
                                                     int(window), base._stream(None)), "fa_mask_plan")


def attention_mask(B: int, N: int, *, documents=None, prefix=None, causal: bool = True, window: int = 0, device=None,
                   stream=None) -> AttentionMask:
    """The mask of attention over B sequences of N rows.

    documents (int32 (B,N)): rows see each other only within a run of equal ids; a row with a
    negative id (padding) sees nothing and is not seen.  causal: key j only for j <= i; prefix
    (int32 (B)): or for j < prefix[b] (needs causal; not with documents or window).  window > 0:
    only keys with i - j < window, and without causal j - i < window."""
    given = documents if documents is not None else prefix
    device = torch.device("cuda") if device is None and given is None else torch.device(device or given.device)
    if device.type != "cuda":
        raise ValueError("attention_mask needs a CUDA device")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    size = fa_mask_plan_size(B, N)
    if size == 0:
        raise base.FAError(2, "attention_mask")
    with launch_on(device, stream) as keep:
        plan = keep(torch.empty(size, device=device, dtype=torch.uint8))
        fa_mask_plan(plan, documents, prefix, B, N, causal, window)
    return AttentionMask(plan, B, N)


# ----------------------------------------------------------------------------- C-ABI calls
def _mod_args(q, k, v, mask, softcap, slopes, causal):
    B, H, N, D = q.shape
    code = dtype_code(q, "q")
    if k.dim() != 4:
        raise ValueError(f"k must be (B,Hkv,N,D), got {tuple(k.shape)}")
    Hkv = k.shape[1]
    base._check(q, "q", q.dtype, (B, H, N, D))
    for name, t in (("k", k), ("v", v)):
        check_on(t, name, q.dtype, (B, Hkv, N, D), q.device)
    if mask is not None:
        if not isinstance(mask, AttentionMask):
            raise TypeError("mask must come from attention_mask")
        if (mask.B, mask.N) != (B, N) or mask.plan.device != q.device:
            raise ValueError(f"mask is for B={mask.B}, N={mask.N} on {mask.plan.device}; "
                             f"q has B={B}, N={N} on {q.device}")
        if causal:
            raise ValueError("causal goes into attention_mask when a mask is given")
    if slopes is not None:
        check_on(slopes, "alibi_slopes", torch.float32, (H,), q.device)
    plan = None if mask is None else base._p(mask.plan)
    return B, H, Hkv, N, D, code, plan


def fa_fwd_mod(q, k, v, o, lse, scale: float, causal: bool, mask=None, softcap: float = 0.0, alibi_slopes=None,
               stream=None) -> None:
    """O, lse <- score-modified attention; q, o (B,H,N,D), k, v (B,Hkv,N,D) bf16 or fp16, lse
    (B,H,N) float32."""
    B, H, Hkv, N, D, code, plan = _mod_args(q, k, v, mask, softcap, alibi_slopes, causal)
    check_on(o, "o", q.dtype, (B, H, N, D), q.device)
    check_on(lse, "lse", torch.float32, (B, H, N), q.device)
    with launch_on(q.device, stream):
        base._raise(base.load_library().fa_fwd_mod(
            base._p(q), base._p(k), base._p(v), base._p(o), base._p(lse), plan, base._p(alibi_slopes), float(softcap),
            B, H, Hkv, N, D, float(scale), int(causal), code, base._stream(None)), "fa_fwd_mod")


def fa_bwd_mod(q, k, v, o, do, lse, dq, dk, dv, workspace, scale: float, causal: bool, mask=None, softcap: float = 0.0,
               alibi_slopes=None, stream=None) -> None:
    """dq, dk, dv <- gradients of fa_fwd_mod; workspace: uint8 CUDA tensor of
    fa_bwd_workspace_size(B, H, N, D) bytes."""
    B, H, Hkv, N, D, code, plan = _mod_args(q, k, v, mask, softcap, alibi_slopes, causal)
    for name, t in (("o", o), ("do", do), ("dq", dq)):
        check_on(t, name, q.dtype, (B, H, N, D), q.device)
    for name, t in (("dk", dk), ("dv", dv)):
        check_on(t, name, q.dtype, (B, Hkv, N, D), q.device)
    check_on(lse, "lse", torch.float32, (B, H, N), q.device)
    wp, wn = base._ws(workspace)
    if workspace.device != q.device:
        raise ValueError(f"workspace must be on {q.device}")
    with launch_on(q.device, stream):
        base._raise(base.load_library().fa_bwd_mod(
            base._p(q), base._p(k), base._p(v), base._p(o), base._p(do), base._p(lse), base._p(dq), base._p(dk),
            base._p(dv), wp, wn, plan, base._p(alibi_slopes), float(softcap), B, H, Hkv, N, D, float(scale),
            int(causal), code, base._stream(None)), "fa_bwd_mod")


# ----------------------------------------------------------------------------- convenience API
def modified(q, k, mask, softcap, alibi_slopes) -> bool:
    """Whether a call needs the score-modified path."""
    return mask is not None or softcap != 0.0 or alibi_slopes is not None or (
        k.dim() == 4 and q.dim() == 4 and k.shape[1] != q.shape[1])


def modified_forward(q, k, v, scale, causal, stream, mask, softcap, alibi_slopes):
    dtype_code(q, "q")
    with launch_on(q.device, stream) as keep:
        o = keep(torch.empty_like(q))
        lse = keep(torch.empty(q.shape[:3], device=q.device, dtype=torch.float32))
        fa_fwd_mod(q, k, v, o, lse, scale, causal, mask, softcap, alibi_slopes)
    return o, lse


def modified_backward(q, k, v, o, lse, do, scale, causal, stream, workspace, mask, softcap, alibi_slopes):
    dtype_code(q, "q")
    with launch_on(q.device, stream) as keep:
        dq, dk, dv = keep(torch.empty_like(q)), keep(torch.empty_like(k)), keep(torch.empty_like(v))
        if workspace is None:
            workspace = torch.empty(base.fa_bwd_workspace_size(*q.shape), device=q.device, dtype=torch.uint8)
        fa_bwd_mod(q, k, v, o, do, lse, dq, dk, dv, workspace, scale, causal, mask, softcap, alibi_slopes)
    return dq, dk, dv


class ModifiedAttention(torch.autograd.Function):
    """autograd wrapper of the score-modified attention."""

    @staticmethod
    def forward(ctx, q, k, v, scale, causal, mask, softcap, alibi_slopes):
        if alibi_slopes is not None and alibi_slopes.requires_grad:
            raise ValueError("alibi_slopes get no gradient; detach them")
        o, lse = modified_forward(q, k, v, scale, causal, None, mask, softcap, alibi_slopes)
        saved = (q, k, v, o, lse) + (() if alibi_slopes is None else (alibi_slopes,))
        ctx.save_for_backward(*saved)
        ctx.args = (scale, causal, mask, softcap)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, *slopes = ctx.saved_tensors
        scale, causal, mask, softcap = ctx.args
        dq, dk, dv = modified_backward(q, k, v, o, lse, do.contiguous(), scale, causal, None, None, mask, softcap,
                                       slopes[0] if slopes else None)
        return dq, dk, dv, None, None, None, None, None
