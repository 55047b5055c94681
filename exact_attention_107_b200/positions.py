"""Rotary positions of queries and keys (argument marshalling for fa_rotary)."""
from __future__ import annotations

import ctypes
import functools
import math

import torch
from torch.autograd.function import once_differentiable

from . import _binding as base
from ._modified import check_on, dtype_code, on, ptr


def rotary_table(length: int, rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None,
                 factor: float = 1.0, original_length: int | None = None, low: float = 1.0, high: float = 32.0,
                 device=None) -> torch.Tensor:
    """(length, rotary_dim) float32 table of the positions 0 .. length-1: cosines, then sines, of
    position * frequency_i, frequency_i = base^(-2i / rotary_dim), computed in 64 bits.

    scaling stretches the frequencies for contexts `factor` times longer than those trained on:
      "linear"    every frequency divided by factor
      "base"      base * factor^(R / (R - 2)): the lowest frequency divided by factor, the highest kept
      "by_parts"  frequencies that turn less than `low` times over original_length divided by factor,
                  those that turn more than `high` times kept, a linear mix in between; cosines and
                  sines times 0.1 ln(factor) + 1, which sharpens the scores of the longer rows"""
    R = int(rotary_dim)
    if length < 1 or R < 2 or R % 2 or not (base > 0 and factor >= 1.0):
        raise ValueError("rotary_table needs length >= 1, an even rotary_dim >= 2, base > 0 and factor >= 1")
    if scaling not in (None, "linear", "base", "by_parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "base":
        if R < 4:
            raise ValueError('scaling "base" needs rotary_dim >= 4')
        base = base * factor ** (R / (R - 2))
    i = torch.arange(0, R, 2, dtype=torch.float64)
    freq = base ** (-i / R)
    size = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if original_length is None or original_length < 1 or not 0 <= low < high:
            raise ValueError('scaling "by_parts" needs original_length >= 1 and 0 <= low < high')
        turns = original_length * freq / (2.0 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        freq = freq * (keep + (1.0 - keep) / factor)
        size = 0.1 * math.log(factor) + 1.0
    angle = torch.arange(length, dtype=torch.float64)[:, None] * freq
    table = (torch.cat([angle.cos(), angle.sin()], 1) * size).float()
    return table if device is None else table.to(device)


def strides3(t: torch.Tensor, name: str):
    """(batch, head, token) strides in elements of a (B,H,N,D) tensor whose D columns are
    contiguous; 0 for axes of size one."""
    shape = t.shape
    b, h, n, d = t.stride()
    if d != 1 and shape[3] > 1:
        raise ValueError(f"{name} must have contiguous columns")
    b, h, n = b if shape[0] > 1 else 0, h if shape[1] > 1 else 0, n if shape[2] > 1 else 0
    if (b | h | n) & 7 or t.data_ptr() & 15:
        raise ValueError(f"{name} must be 16-byte aligned, with batch, head and token strides that are multiples "
                         f"of 8 elements; got strides {tuple(t.stride())}")
    return b, h, n


@functools.lru_cache(maxsize=256)
def c_strides(s):
    return (ctypes.c_longlong * 3)(*s)


def check_strided(t, name, dtype, shape, device) -> None:
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def check_table(table, D, device):
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a (positions, rotary columns) tensor, as rotary_table makes it")
    check_on(table, "table", torch.float32, table.shape, device)
    rows, R = table.shape
    if R < 2 or R % 2 or R > D or rows < 1:
        raise ValueError(f"table must have an even number of columns from 2 to {D} and a row, got {tuple(table.shape)}")
    return R


def _rotary_args(q, k, table, positions):
    """Checks the inputs; returns (shape, heads, strides, the C call's middle arguments)."""
    some = q if q is not None else k
    if some is None:
        raise ValueError("q and k cannot both be None")
    code = dtype_code(some, "q" if q is not None else "k")
    if some.dim() != 4:
        raise ValueError(f"q and k must be (B,H,N,D), got {tuple(some.shape)}")
    B, _, N, D = some.shape
    dev, dtype = some.device, some.dtype
    H = Hkv = 0
    qs = ks = None
    if q is not None:
        H = q.shape[1]
        qs = c_strides(strides3(q, "q"))
    if k is not None:
        Hkv = k.shape[1] if k.dim() == 4 else 0
        check_strided(k, "k", dtype, (B, Hkv, N, D), dev)
        ks = c_strides(strides3(k, "k"))
    R = check_table(table, D, dev)
    stride = 0
    if positions is not None:
        if not isinstance(positions, torch.Tensor):
            raise TypeError("positions must be a torch.Tensor")
        shape = (N,) if positions.dim() == 1 else ((1, N) if positions.shape == (1, N) else (B, N))
        check_on(positions, "positions", torch.int32, shape, dev)
        stride = N if shape == (B, N) and B > 1 else 0
    return B, H, Hkv, N, D, R, code, dev, (ptr(positions), qs, ks, stride, table.shape[0])


def _rotary(raw, keep, q, k, q_out, k_out, table, middle, tail):
    base._raise(base.load_library().fa_rotary(ptr(q), ptr(k), ptr(q_out), ptr(k_out), table.data_ptr(), *middle, *tail,
                                              raw), "fa_rotary")


def fa_rotary(q, k, q_out, k_out, table, positions=None, interleaved: bool = False, inverse: bool = False,
              stream=None) -> None:
    """q_out, k_out <- q, k (bf16 or fp16 (B,H,N,D) and (B,Hkv,N,D), k or q None to leave it out)
    with each row turned by its position; inverse turns back.  Inputs may be strided; outputs are
    contiguous.  positions: int32 (N), (1,N) or (B,N), None: 0 .. N-1."""
    B, H, Hkv, N, D, R, code, dev, middle = _rotary_args(q, k, table, positions)
    dtype = (q if q is not None else k).dtype
    if q is not None:
        check_on(q_out, "q_out", dtype, (B, H, N, D), dev)
    if k is not None:
        check_on(k_out, "k_out", dtype, (B, Hkv, N, D), dev)
    on(dev, stream, _rotary, q, k, q_out if q is not None else None, k_out if k is not None else None, table, middle,
       (B, H, Hkv, N, D, R, int(interleaved), int(inverse), code))


def _turn(q, k, table, positions, interleaved, inverse, stream):
    if base.fast_path(stream):
        r = base.fast_result(base._fast.rotary(q, k, table, positions, interleaved, inverse), "fa_rotary")
        if r is not None:
            return r
    B, H, Hkv, N, D, R, code, dev, middle = _rotary_args(q, k, table, positions)
    tail = (B, H, Hkv, N, D, R, int(interleaved), int(inverse), code)

    def call(raw, keep):
        q_out = None if q is None else keep(q.new_empty(q.shape))
        k_out = None if k is None else keep(k.new_empty(k.shape))
        _rotary(raw, keep, q, k, q_out, k_out, table, middle, tail)
        return q_out, k_out

    return on(dev, stream, call)


def rotary_forward(q, k, table, *, positions=None, interleaved: bool = False, stream=None):
    """Returns (q, k) with the first R columns of each row turned by its position: table
    (positions, R) from rotary_table; pairs are columns (i, i + R/2), or (2i, 2i + 1) when
    interleaved.  Either tensor may be None.  positions: int32 (N), (1,N) or (B,N), None: 0 .. N-1;
    a position outside the table leaves its row unturned and sets the device status
    (fa_device_status) to FA_ERR_INDEX."""
    return _turn(q, k, table, positions, interleaved, False, stream)


def rotary_backward(dq, dk, table, *, positions=None, interleaved: bool = False, stream=None):
    """Returns the gradients of rotary_forward's inputs from those of its outputs."""
    return _turn(dq, dk, table, positions, interleaved, True, stream)


def _readable(t):
    """t, or a contiguous copy where its strides are not ones that the kernel reads."""
    if t is None:
        return None
    try:
        strides3(t, "gradient")
        return t
    except ValueError:
        return t.contiguous()


class RotaryEmbedding(torch.autograd.Function):
    """autograd wrapper of rotary_forward / rotary_backward.  Under CUDA graph capture the rule of
    ModifiedAttention holds."""

    @staticmethod
    def forward(ctx, q, k, table, positions, interleaved):
        if table.requires_grad:
            raise ValueError("the table gets no gradient; detach it")
        ctx.save_for_backward(*((table,) if positions is None else (table, positions)))
        ctx.interleaved = interleaved
        return rotary_forward(q, k, table, positions=positions, interleaved=interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        table, *positions = ctx.saved_tensors
        if dq is None and dk is None:
            return None, None, None, None, None
        dq, dk = rotary_backward(_readable(dq), _readable(dk), table, positions=positions[0] if positions else None,
                                 interleaved=ctx.interleaved)
        return dq, dk, None, None, None


def rotary_embedding(q, k, table, *, positions=None, interleaved: bool = False):
    """Differentiable rotary_forward."""
    return RotaryEmbedding.apply(q, k, table, positions, interleaved)
