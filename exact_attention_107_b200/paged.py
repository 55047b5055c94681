"""Paged key-value cache: appending new tokens and attending to it (argument marshalling for
fa_paged_append and fa_paged_attention).

A cache is two pools of pages, k_pages and v_pages (num_pages, Hkv, page_size, D) with page_size a
power of two from 8 to 256, an int32 block_table (B, width) that gives each sequence its pages in
order, and int32 seq_lens (B), which count the new tokens of the current step."""
from __future__ import annotations

import functools

import torch

from . import _binding as base
from ._modified import check_on, dtype_code, on, ptr
from .positions import c_strides, check_strided, check_table, strides3


def _check_cache(k_pages, v_pages, block_table, seq_lens, dtype, B, D, device):
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be (num_pages, Hkv, page_size, D)")
    num_pages, Hkv, page, _ = shape = k_pages.shape
    if shape[3] != D:
        raise ValueError(f"k_pages must have {D} columns, got {tuple(shape)}")
    check_on(k_pages, "k_pages", dtype, shape, device)
    check_on(v_pages, "v_pages", dtype, shape, device)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be (B, pages per sequence)")
    width = block_table.shape[1]
    check_on(block_table, "block_table", torch.int32, (B, width), device)
    check_on(seq_lens, "seq_lens", torch.int32, (B,), device)
    return num_pages, Hkv, page, width


def _append_args(k, v, k_pages, v_pages, q, block_table, seq_lens, new_lens, table):
    code = dtype_code(k, "k")
    if k.dim() != 4:
        raise ValueError(f"k must be (B,Hkv,T,D), got {tuple(k.shape)}")
    B, Hkv, T, D = k.shape
    dev, dtype = k.device, k.dtype
    check_strided(v, "v", dtype, (B, Hkv, T, D), dev)
    num_pages, heads, page, width = _check_cache(k_pages, v_pages, block_table, seq_lens, dtype, B, D, dev)
    if heads != Hkv:
        raise ValueError(f"k has {Hkv} heads, the pages {heads}")
    H, qs = 0, None
    if q is not None:
        H = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 4 else 0
        check_strided(q, "q", dtype, (B, H, T, D), dev)
        qs = c_strides(strides3(q, "q"))
    if new_lens is not None:
        check_on(new_lens, "new_lens", torch.int32, (B,), dev)
    R = rows = 0
    if table is not None:
        R, rows = check_table(table, D, dev), table.shape[0]
    return (B, H, T, D), (c_strides(strides3(k, "k")), c_strides(strides3(v, "v")), qs, rows, width, num_pages, page,
                          B, H, Hkv, T, D, R), code


def _append(raw, keep, k, v, k_pages, v_pages, q, q_out, block_table, seq_lens, new_lens, table, args, interleaved, code):
    base._raise(base.load_library().fa_paged_append(
        k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), ptr(q), ptr(q_out), block_table.data_ptr(),
        seq_lens.data_ptr(), ptr(new_lens), ptr(table), *args, int(interleaved), code, raw), "fa_paged_append")


def fa_paged_append(k, v, k_pages, v_pages, q, q_out, block_table, seq_lens, new_lens=None, table=None,
                    interleaved: bool = False, stream=None) -> None:
    """The pages <- k (turned when a table is given), v; q_out <- q turned (q None: left out).
    Arguments as paged_append; q_out contiguous."""
    shape, args, code = _append_args(k, v, k_pages, v_pages, q, block_table, seq_lens, new_lens, table)
    if q is not None:
        check_on(q_out, "q_out", k.dtype, shape, k.device)
    on(k.device, stream, _append, k, v, k_pages, v_pages, q, q_out if q is not None else None, block_table, seq_lens,
       new_lens, table, args, interleaved, code)


def paged_append(k, v, k_pages, v_pages, block_table, seq_lens, *, new_lens=None, q=None, table=None,
                 interleaved: bool = False, stream=None):
    """Writes the keys and values (B,Hkv,T,D) of new tokens into their sequences' pages, in place.

    Token t of sequence b takes position seq_lens[b] - n + t with n = new_lens[b] (int32 (B), 0 to
    T; None: T; a count outside that writes nothing and sets the status as below); rows t >= n are not
    written.  With a table (rotary_table) the keys are turned by
    their positions, and so is q (B,H,T,D), whose turned copy is returned (None without q; rows
    t >= n are zero).  k, v and q may be strided.  Two rows that fall on the same slot (sequences
    that share the page being written) leave a mix of the two there.  A token without a page, or with
    a table one whose position the table does not hold, is not written, neither its key nor its value;
    it sets the device status (fa_device_status) to FA_ERR_INDEX.  A row of q whose position the table
    does not hold comes back unturned."""
    if table is None and q is not None:
        raise ValueError("q is turned on the way and needs a table")
    if base.fast_path(stream):
        r = base.fast_result(base._fast.append(k, v, k_pages, v_pages, block_table, seq_lens, new_lens, q, table,
                                               interleaved), "fa_paged_append")
        if r is not None:
            return r[0]
    shape, args, code = _append_args(k, v, k_pages, v_pages, q, block_table, seq_lens, new_lens, table)

    def call(raw, keep):
        q_out = None if q is None else keep(q.new_empty(shape))
        _append(raw, keep, k, v, k_pages, v_pages, q, q_out, block_table, seq_lens, new_lens, table, args, interleaved,
                code)
        return q_out

    return on(k.device, stream, call)


@functools.lru_cache(maxsize=256)
def fa_paged_workspace_size(B: int, H: int, Hkv: int, T: int, D: int) -> int:
    return int(base.load_library().fa_paged_workspace_size(B, H, Hkv, T, D))


def _decode_args(q, k_pages, v_pages, block_table, seq_lens, alibi_slopes):
    code = dtype_code(q, "q")
    if q.dim() != 4:
        raise ValueError(f"q must be (B,H,T,D), got {tuple(q.shape)}")
    B, H, T, D = q.shape
    dev = q.device
    check_on(q, "q", q.dtype, q.shape, dev)
    num_pages, Hkv, page, width = _check_cache(k_pages, v_pages, block_table, seq_lens, q.dtype, B, D, dev)
    if alibi_slopes is not None:
        check_on(alibi_slopes, "alibi_slopes", torch.float32, (H,), dev)
    return (width, num_pages, page, B, H, Hkv, T, D), code


def _decode(raw, keep, q, k_pages, v_pages, block_table, seq_lens, o, lse, workspace, alibi_slopes, softcap, window,
            args, scale, code):
    base._raise(base.load_library().fa_paged_attention(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        ptr(alibi_slopes), float(softcap), int(window), *args, float(scale), code, raw), "fa_paged_attention")


def _check_workspace(workspace, dev):
    base._ws(workspace)
    if workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}")


def fa_paged_attention(q, k_pages, v_pages, block_table, seq_lens, o, lse, workspace, scale: float,
                       softcap: float = 0.0, alibi_slopes=None, window: int = 0, stream=None) -> None:
    """o, lse <- paged_attention; o (B,H,T,D), lse (B,H,T) float32, workspace of
    fa_paged_workspace_size bytes (one for each call that may overlap)."""
    args, code = _decode_args(q, k_pages, v_pages, block_table, seq_lens, alibi_slopes)
    check_on(o, "o", q.dtype, q.shape, q.device)
    check_on(lse, "lse", torch.float32, q.shape[:3], q.device)
    _check_workspace(workspace, q.device)
    on(q.device, stream, _decode, q, k_pages, v_pages, block_table, seq_lens, o, lse, workspace, alibi_slopes, softcap,
       window, args, scale, code)


def paged_attention(q, k_pages, v_pages, block_table, seq_lens, scale: float | None = None, *, softcap: float = 0.0,
                    alibi_slopes=None, window: int = 0, workspace=None, stream=None):
    """Returns (O, lse): causal attention of the last T tokens (1 to 64) of each sequence over its
    cached keys and values, which already hold them (paged_append).

    q (B,H,T,D), H a multiple of the pages' Hkv.  Row t of sequence b has position p =
    seq_lens[b] - T + t and sees keys j <= p, with window > 0 those with p - j < window; a row with
    p < 0 has O = 0 and lse = -inf.  softcap and alibi_slopes as in attention_forward, so that a
    model trained there (head dims up to 128 with these) is served here; this call takes 256 columns
    too.  Table entries past a sequence's last page, or wholly before
    every row's window, are not read; a page outside the pool counts as absent and sets the device
    status (fa_device_status) to FA_ERR_INDEX.  workspace: for callers that keep one, of
    fa_paged_workspace_size bytes; calls that may overlap on the GPU (other streams, captured
    graphs) must not share it."""
    if scale is None and isinstance(q, torch.Tensor) and q.dim() == 4:
        scale = base.default_scale(q.shape[3])
    if base.fast_path(stream) and workspace is None:
        r = base.fast_result(base._fast.decode(q, k_pages, v_pages, block_table, seq_lens, scale, softcap,
                                               alibi_slopes, window), "fa_paged_attention")
        if r is not None:
            return r
    args, code = _decode_args(q, k_pages, v_pages, block_table, seq_lens, alibi_slopes)
    if workspace is not None:
        _check_workspace(workspace, q.device)

    def call(raw, keep):
        o, lse = keep(torch.empty_like(q)), keep(q.new_empty(q.shape[:3], dtype=torch.float32))
        ws = workspace
        if ws is None:
            ws = q.new_empty(max(16, fa_paged_workspace_size(*args[3:])), dtype=torch.uint8)
        _decode(raw, keep, q, k_pages, v_pages, block_table, seq_lens, o, lse, ws, alibi_slopes, softcap, window, args,
                scale, code)
        return o, lse

    return on(q.device, stream, call)
