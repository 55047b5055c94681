"""Score-modified attention: shared key-value heads, interval masks, capped scores and a distance
bias (argument marshalling for fa_mask_plan, fa_fwd_mod and fa_bwd_mod)."""
from __future__ import annotations

import contextlib

import torch
from torch.autograd.function import once_differentiable

from . import _binding as base

DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1}
# Not there in a torch without CUDA, where no call gets as far as to need them.
_device_now = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def stream_here(device, stream):
    """The raw current stream where a call may launch as it is: no stream given and `device` current.
    Otherwise None, and the call goes through launch_on."""
    if stream is None and _device_now() == device.index:
        return _raw_stream(device.index)
    return None


@contextlib.contextmanager
def launch_on(device, stream):
    """Makes `device` and `stream` (None: the device's current stream; a torch.cuda.Stream or a raw
    cudaStream_t) current, so that what a call allocates belongs to the stream its kernels run on.
    Yields the raw stream and a function that registers an output for use on the caller's own
    stream too."""
    caller = torch.cuda.current_stream(device)
    if stream is None:
        stream = caller
    elif not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")

    def keep(t):
        if t is not None and stream != caller:
            t.record_stream(caller)
        return t

    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield stream.cuda_stream, keep


def no_keep(t):
    return t


def on(device, stream, call, *args):
    """call(raw stream, keep, *args), launched on `device` and `stream`."""
    raw = stream_here(device, stream)
    if raw is not None:
        return call(raw, no_keep, *args)
    with launch_on(device, stream) as (raw, keep):
        return call(raw, keep, *args)


def check_on(t, name, dtype, shape, device) -> None:
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    base._check(t, name, dtype, shape)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def dtype_code(t, name) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float16, got {t.dtype}")
    return code


def ptr(t):
    return None if t is None else t.data_ptr()


# ----------------------------------------------------------------------------- masks
class AttentionMask:
    """Which keys each row may see, for B batch elements of N rows: the plan of fa_mask_plan on
    its device.  Made by attention_mask; any number of calls may use it, on any stream that runs
    after the one it was made on, and it may be dropped as soon as the last of them has returned."""

    def __init__(self, plan: torch.Tensor, B: int, N: int, raw=None):
        self.plan, self.B, self.N = plan, B, N
        self._known = {raw}                      # raw streams that the plan's memory is kept for

    def used_on(self, raw) -> None:
        """Keeps the plan's memory from being handed out again before what runs on the stream now has
        read it: callers hold a mask, not its memory, so they cannot do it."""
        if raw not in self._known:
            self.plan.record_stream(torch.cuda.ExternalStream(raw, device=self.plan.device))
            self._known.add(raw)


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
    on(plan.device, stream, _mask_plan, pp, pn, documents, prefix, B, N, causal, window)


def _mask_plan(raw, keep, pp, pn, documents, prefix, B, N, causal, window):
    base._raise(base.load_library().fa_mask_plan(pp, pn, ptr(documents), ptr(prefix), B, N, int(causal), int(window),
                                                 raw), "fa_mask_plan")


def _new_plan(raw, keep, device, size):
    return keep(torch.empty(size, device=device, dtype=torch.uint8)), raw


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
    if base.fast_path(stream):
        r = base.fast_result(base._fast.mask_plan(documents, prefix, B, N, causal, window, device.index), "fa_mask_plan")
        if r is not None:
            return AttentionMask(r[0], B, N, _raw_stream(device.index))
    size = fa_mask_plan_size(B, N)
    if size == 0:
        raise base.FAError(2, "fa_mask_plan")
    plan, raw = on(device, stream, _new_plan, device, size)
    fa_mask_plan(plan, documents, prefix, B, N, causal, window, stream)
    return AttentionMask(plan, B, N, raw)


# ----------------------------------------------------------------------------- C-ABI calls
def _mod_args(q, k, v, mask, softcap, slopes, causal):
    """Checks what forward and backward share; returns the C call's tail up to the stream."""
    code = dtype_code(q, "q")
    if q.dim() != 4:
        raise ValueError(f"q must be (B,H,N,D), got {tuple(q.shape)}")
    B, H, N, D = q.shape
    dev, dtype = q.device, q.dtype
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be (B,Hkv,N,D)")
    Hkv = k.shape[1]
    check_on(q, "q", dtype, (B, H, N, D), dev)
    check_on(k, "k", dtype, (B, Hkv, N, D), dev)
    check_on(v, "v", dtype, (B, Hkv, N, D), dev)
    plan = None
    if mask is not None:
        if not isinstance(mask, AttentionMask):
            raise TypeError("mask must come from attention_mask")
        if mask.B != B or mask.N != N or mask.plan.device != dev:
            raise ValueError(f"mask is for B={mask.B}, N={mask.N} on {mask.plan.device}; q has B={B}, N={N} on {dev}")
        if causal:
            raise ValueError("causal goes into attention_mask when a mask is given")
        plan = mask.plan.data_ptr()
    if slopes is not None:
        check_on(slopes, "alibi_slopes", torch.float32, (H,), dev)
    return B, H, Hkv, N, D, code, (plan, ptr(slopes), float(softcap), B, H, Hkv, N, D)


def fa_fwd_mod(q, k, v, o, lse, scale: float, causal: bool, mask=None, softcap: float = 0.0, alibi_slopes=None,
               stream=None) -> None:
    """O, lse <- score-modified attention; q, o (B,H,N,D), k, v (B,Hkv,N,D) bf16 or fp16, lse
    (B,H,N) float32."""
    B, H, _, N, D, code, mods = _mod_args(q, k, v, mask, softcap, alibi_slopes, causal)
    check_on(o, "o", q.dtype, (B, H, N, D), q.device)
    check_on(lse, "lse", torch.float32, (B, H, N), q.device)
    on(q.device, stream, _fwd, q, k, v, o, lse, mask, mods, scale, causal, code)


def _fwd(raw, keep, q, k, v, o, lse, mask, mods, scale, causal, code):
    if mask is not None:
        mask.used_on(raw)
    base._raise(base.load_library().fa_fwd_mod(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                               *mods, float(scale), int(causal), code, raw), "fa_fwd_mod")


def fa_bwd_mod(q, k, v, o, do, lse, dq, dk, dv, workspace, scale: float, causal: bool, mask=None, softcap: float = 0.0,
               alibi_slopes=None, stream=None) -> None:
    """dq, dk, dv <- gradients of fa_fwd_mod; workspace: uint8 CUDA tensor of
    fa_bwd_workspace_size(B, H, N, D) bytes."""
    B, H, Hkv, N, D, code, mods = _mod_args(q, k, v, mask, softcap, alibi_slopes, causal)
    _check_grads(q, o, do, lse, B, H, N, D)
    check_on(dq, "dq", q.dtype, (B, H, N, D), q.device)
    check_on(dk, "dk", q.dtype, (B, Hkv, N, D), q.device)
    check_on(dv, "dv", q.dtype, (B, Hkv, N, D), q.device)
    base._ws(workspace)
    if workspace.device != q.device:
        raise ValueError(f"workspace must be on {q.device}")
    on(q.device, stream, _bwd, q, k, v, o, do, lse, dq, dk, dv, workspace, mask, mods, scale, causal, code)


def _check_grads(q, o, do, lse, B, H, N, D):
    check_on(o, "o", q.dtype, (B, H, N, D), q.device)
    check_on(do, "do", q.dtype, (B, H, N, D), q.device)
    check_on(lse, "lse", torch.float32, (B, H, N), q.device)


def _bwd(raw, keep, q, k, v, o, do, lse, dq, dk, dv, workspace, mask, mods, scale, causal, code):
    if mask is not None:
        mask.used_on(raw)
    base._raise(base.load_library().fa_bwd_mod(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(), dq.data_ptr(),
        dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), *mods,
        float(scale), int(causal), code, raw), "fa_bwd_mod")


# ----------------------------------------------------------------------------- convenience API
def modified(q, k, mask, softcap, alibi_slopes) -> bool:
    """Whether a call needs the score-modified path."""
    return mask is not None or softcap != 0.0 or alibi_slopes is not None or (
        k.dim() == 4 and q.dim() == 4 and k.shape[1] != q.shape[1])


def _fits(mask, q):
    """Whether a call may go to _fast with this mask, which is then kept for the current stream."""
    if mask is None:
        return True
    if not (isinstance(mask, AttentionMask) and q.shape[0] == mask.B and q.shape[2] == mask.N):
        return False
    mask.used_on(_raw_stream(mask.plan.device.index))
    return True


def modified_forward(q, k, v, scale, causal, stream, mask, softcap, alibi_slopes):
    if base.fast_path(stream) and _fits(mask, q):
        r = base.fast_result(base._fast.forward(q, k, v, None if mask is None else mask.plan, alibi_slopes, softcap,
                                                scale, causal), "fa_fwd_mod")
        if r is not None:
            return r
    _, _, _, _, _, code, mods = _mod_args(q, k, v, mask, softcap, alibi_slopes, causal)

    def call(raw, keep):
        o, lse = keep(torch.empty_like(q)), keep(q.new_empty(q.shape[:3], dtype=torch.float32))
        _fwd(raw, keep, q, k, v, o, lse, mask, mods, scale, causal, code)
        return o, lse

    return on(q.device, stream, call)


def modified_backward(q, k, v, o, lse, do, scale, causal, stream, workspace, mask, softcap, alibi_slopes):
    if base.fast_path(stream) and workspace is None and _fits(mask, q):
        r = base.fast_result(base._fast.backward(q, k, v, None if mask is None else mask.plan, alibi_slopes, softcap,
                                                 scale, causal, o, lse, do), "fa_bwd_mod")
        if r is not None:
            return r
    B, H, Hkv, N, D, code, mods = _mod_args(q, k, v, mask, softcap, alibi_slopes, causal)
    _check_grads(q, o, do, lse, B, H, N, D)
    if workspace is not None:
        base._ws(workspace)
        if workspace.device != q.device:
            raise ValueError(f"workspace must be on {q.device}")

    def call(raw, keep):
        grads = [keep(torch.empty_like(t)) for t in (q, k, v)]
        ws = workspace
        if ws is None:
            ws = q.new_empty(base.fa_bwd_workspace_size(B, H, N, D), dtype=torch.uint8)
        _bwd(raw, keep, q, k, v, o, do, lse, *grads, ws, mask, mods, scale, causal, code)
        return tuple(grads)

    return on(q.device, stream, call)


class ModifiedAttention(torch.autograd.Function):
    """autograd wrapper of the score-modified attention.  Under CUDA graph capture torch's own rule
    holds: no autograd graph of the same leaves made outside the capture may be alive; the functional
    calls (attention_forward, attention_backward) have no such rule."""

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
