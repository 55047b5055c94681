"""Paged key-value cache: appending new tokens and attending to it (argument marshalling for
fa_paged_append and fa_paged_attention).

A cache is two pools of pages, k_pages and v_pages (num_pages, Hkv, page_size, D) with page_size a
power of two from 8 to 256, an int32 block_table (B, width) that gives each sequence its pages in
order, and int32 seq_lens (B), which count the new tokens of the current step."""
from __future__ import annotations

import torch

from . import _binding as base
from ._modified import check_on, dtype_code, launch_on
from .positions import c_strides, check_strided, check_table, strides3


def _check_cache(k_pages, v_pages, block_table, seq_lens, dtype, B, D, device):
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be (num_pages, Hkv, page_size, D)")
    num_pages, Hkv, page, _ = k_pages.shape
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        check_on(t, name, dtype, (num_pages, Hkv, page, D), device)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be (B, pages per sequence)")
    check_on(block_table, "block_table", torch.int32, (B, block_table.shape[1]), device)
    check_on(seq_lens, "seq_lens", torch.int32, (B,), device)
    return num_pages, Hkv, page, block_table.shape[1]


def fa_paged_append(k, v, k_pages, v_pages, q, q_out, block_table, seq_lens, new_lens=None, table=None,
                    interleaved: bool = False, stream=None) -> None:
    """The pages <- k (turned when a table is given), v; q_out <- q turned (q None: left out).
    Arguments as paged_append; q_out contiguous."""
    code = dtype_code(k, "k")
    if k.dim() != 4:
        raise ValueError(f"k must be (B,Hkv,T,D), got {tuple(k.shape)}")
    B, Hkv, T, D = k.shape
    dev = k.device
    check_strided(v, "v", k.dtype, (B, Hkv, T, D), dev)
    num_pages, heads, page, width = _check_cache(k_pages, v_pages, block_table, seq_lens, k.dtype, B, D, dev)
    if heads != Hkv:
        raise ValueError(f"k has {Hkv} heads, the pages {heads}")
    H, qs = 0, None
    if q is not None:
        H = q.shape[1] if q.dim() == 4 else 0
        check_strided(q, "q", k.dtype, (B, H, T, D), dev)
        check_on(q_out, "q_out", k.dtype, (B, H, T, D), dev)
        qs = c_strides(strides3(q, "q"))
    if new_lens is not None:
        check_on(new_lens, "new_lens", torch.int32, (B,), dev)
    R = 0 if table is None else check_table(table, D, dev)
    with launch_on(dev, stream):
        base._raise(base.load_library().fa_paged_append(
            base._p(k), base._p(v), base._p(k_pages), base._p(v_pages), base._p(q),
            base._p(q_out if q is not None else None), base._p(block_table), base._p(seq_lens), base._p(new_lens),
            base._p(table), c_strides(strides3(k, "k")), c_strides(strides3(v, "v")), qs,
            0 if table is None else table.shape[0], width, num_pages, page, B, H, Hkv, T, D, R, int(interleaved), code,
            base._stream(None)), "fa_paged_append")


def paged_append(k, v, k_pages, v_pages, block_table, seq_lens, *, new_lens=None, q=None, table=None,
                 interleaved: bool = False, stream=None):
    """Writes the keys and values (B,Hkv,T,D) of new tokens into their sequences' pages, in place.

    Token t of sequence b takes position seq_lens[b] - n + t with n = new_lens[b] (int32 (B), 0 to
    T; None: T); rows t >= n are not written.  With a table (rotary_table) the keys are turned by
    their positions, and so is q (B,H,T,D), whose turned copy is returned (None without q; rows
    t >= n are zero).  k, v and q may be strided.  Two rows that fall on the same slot (sequences
    that share the page being written) leave either's values there.  A page or position outside its
    table is not written and sets the device status (fa_device_status) to FA_ERR_INDEX."""
    if table is None and q is not None:
        raise ValueError("q is turned on the way and needs a table")
    dtype_code(k, "k")
    with launch_on(k.device, stream) as keep:
        q_out = None if q is None else keep(torch.empty(q.shape, device=q.device, dtype=q.dtype))
        fa_paged_append(k, v, k_pages, v_pages, q, q_out, block_table, seq_lens, new_lens, table, interleaved)
    return q_out


def fa_paged_workspace_size(B: int, H: int, Hkv: int, T: int, D: int) -> int:
    return int(base.load_library().fa_paged_workspace_size(B, H, Hkv, T, D))


def fa_paged_attention(q, k_pages, v_pages, block_table, seq_lens, o, lse, workspace, scale: float,
                       softcap: float = 0.0, alibi_slopes=None, window: int = 0, stream=None) -> None:
    """o, lse <- paged_attention; o (B,H,T,D), lse (B,H,T) float32, workspace of
    fa_paged_workspace_size bytes (one for each call that may overlap)."""
    code = dtype_code(q, "q")
    if q.dim() != 4:
        raise ValueError(f"q must be (B,H,T,D), got {tuple(q.shape)}")
    B, H, T, D = q.shape
    dev = q.device
    base._check(q, "q", q.dtype, (B, H, T, D))
    num_pages, Hkv, page, width = _check_cache(k_pages, v_pages, block_table, seq_lens, q.dtype, B, D, dev)
    check_on(o, "o", q.dtype, (B, H, T, D), dev)
    check_on(lse, "lse", torch.float32, (B, H, T), dev)
    if alibi_slopes is not None:
        check_on(alibi_slopes, "alibi_slopes", torch.float32, (H,), dev)
    wp, wn = base._ws(workspace)
    if workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}")
    with launch_on(dev, stream):
        base._raise(base.load_library().fa_paged_attention(
            base._p(q), base._p(k_pages), base._p(v_pages), base._p(block_table), base._p(seq_lens), base._p(o),
            base._p(lse), wp, wn, base._p(alibi_slopes), float(softcap), int(window), width, num_pages, page,
            B, H, Hkv, T, D, float(scale), code, base._stream(None)), "fa_paged_attention")


def paged_attention(q, k_pages, v_pages, block_table, seq_lens, scale: float | None = None, *, softcap: float = 0.0,
                    alibi_slopes=None, window: int = 0, workspace=None, stream=None):
    """Returns (O, lse): causal attention of the last T tokens (1 to 64) of each sequence over its
    cached keys and values, which already hold them (paged_append).

    q (B,H,T,D), H a multiple of the pages' Hkv.  Row t of sequence b has position p =
    seq_lens[b] - T + t and sees keys j <= p, with window > 0 those with p - j < window; a row with
    p < 0 has O = 0 and lse = -inf.  softcap and alibi_slopes as in attention_forward, so that a
    model trained there is served here.  Table entries past a sequence's last page are not read; a
    page outside the pool counts as absent and sets the device status (fa_device_status) to
    FA_ERR_INDEX.  workspace: for callers that keep one, of fa_paged_workspace_size bytes; calls
    that may overlap on the GPU (other streams, captured graphs) must not share it."""
    dtype_code(q, "q")
    if q.dim() != 4 or not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("q must be (B,H,T,D) and k_pages (num_pages, Hkv, page_size, D)")
    B, H, T, D = q.shape
    scale = base.default_scale(D) if scale is None else scale
    with launch_on(q.device, stream) as keep:
        o = keep(torch.empty(q.shape, device=q.device, dtype=q.dtype))
        lse = keep(torch.empty(B, H, T, device=q.device, dtype=torch.float32))
        if workspace is None:
            workspace = torch.empty(max(16, fa_paged_workspace_size(B, H, k_pages.shape[1], T, D)), device=q.device,
                                    dtype=torch.uint8)
        fa_paged_attention(q, k_pages, v_pages, block_table, seq_lens, o, lse, workspace, scale, softcap,
                           alibi_slopes, window)
    return o, lse
