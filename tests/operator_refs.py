"""Plain 64-bit forms of the rotary, paged-cache and score-modified operators, with elementwise
bounds on what the kernels may be off by (tests only).

Bounds are sums of the roundings that a kernel makes, u = finfo(dtype).eps / 2 for one rounding to
the 16-bit type (`tiny` = half its smallest step, for values below its normal range):
  scores       E = 2^-20 (|q|.|k| scale + 1) + 2^-20 cap: products of 16-bit values are exact, the
               tensor core's fp32 sums over up to 256 columns and the fp32 steps after them are
               below that; capped scores carry 2 cap times sigma's error (2^-22)
  P            relative 2 E + 2^-20 against the row's sum, and one rounding u (absolute `tiny`)
  O            sum_j |dP_j| |v_j| + u |O|
  delta        |dO| . |dO's O error| + fp32 sums
  dS           P's error times |dP - delta|, P times the error of (dP - delta), one more rounding
  gradients    the above against |K|, |Q|, |dO|, and their own rounding u
"""
from __future__ import annotations

import math

import torch

F = 2.0 ** -20
NEG = float("-inf")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134


def visible(B, N, documents=None, prefix=None, causal=True, window=0):
    """(B, N, N) bool by the definition, pair by pair."""
    out = torch.zeros(B, N, N, dtype=torch.bool)
    for b in range(B):
        i = torch.arange(N)[:, None]
        j = torch.arange(N)[None, :]
        ok = torch.ones(N, N, dtype=torch.bool)
        if documents is not None:
            ids = documents[b].tolist()
            run, runs = 0, []
            for n in range(N):
                run += int(n > 0 and ids[n] != ids[n - 1])
                runs.append(run)
            r = torch.tensor(runs)
            ok = (r[:, None] == r[None, :]) & (documents[b] >= 0)[:, None]
        if causal:
            near = j <= i
            if prefix is not None:
                near = near | (j < int(prefix[b]))
            ok = ok & near
        if window > 0:
            ok = ok & (i - j < window)
            if not causal:
                ok = ok & (j - i < window)
        out[b] = ok
    return out


def attention(q, k, v, do, scale, seen, softcap=0.0, slopes=None):
    """(values, bounds): dicts of O, lse and, with do, dQ, dK, dV, in float64 on the CPU."""
    dtype = q.dtype
    u, t16 = half_step(dtype), tiny(dtype)
    q, k, v = (x.double().cpu() for x in (q, k, v))
    B, H, N, D = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = scale * q @ kk.transpose(-1, -2)
    e = F * (scale * q.abs() @ kk.abs().transpose(-1, -2) + 1.0)
    x, bend = s, torch.ones_like(s)
    if softcap:
        th = torch.tanh(s / softcap)
        x, bend = softcap * th, 1.0 - th * th
        e = e + F * softcap
    if slopes is not None:
        i = torch.arange(N, dtype=torch.float64)
        bias = slopes.double().cpu().view(1, H, 1, 1) * (i[:, None] - i[None, :]).abs()
        x = x - bias
        e = e + F * bias
    seen = seen.view(B, 1, N, N)
    x = x.masked_fill(~seen, NEG)
    e = e.masked_fill(~seen, 0.0)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse == NEG, 0.0, lse)[..., None])
    O = p @ vv
    row_e = e.amax(-1)
    dp_rel = 2.0 * row_e[..., None] + F                    # of P, against its row
    dp = p * (dp_rel + u) + torch.where(seen, t16, 0.0)
    dO_ = dp @ vv.abs() + (u + F) * O.abs() + t16
    val = {"O": O, "lse": lse}
    bnd = {"O": dO_, "lse": row_e + F * (1.0 + torch.where(lse == NEG, 0.0, lse.abs()))}
    if do is None:
        return val, bnd
    do = do.double().cpu()
    g = do @ vv.transpose(-1, -2)
    ge = F * (do.abs() @ vv.abs().transpose(-1, -2))
    delta = (do * O).sum(-1, keepdim=True)
    de = (do.abs() * (dO_ + F * O.abs())).sum(-1, keepdim=True)
    w = p * bend
    we = p * F + w * (2.0 * dp_rel + u) + torch.where(seen, t16, 0.0)      # P from the rounded lse
    ds = w * (g - delta)
    dse = we * (g - delta).abs() + (w + we) * (ge + de) + u * ds.abs() + torch.where(seen, t16, 0.0)
    dse = dse * (1.0 + u)
    shared = lambda y: y.view(B, Hkv, G, N, D).sum(2)
    dQ, dQe = scale * ds @ kk, scale * dse @ kk.abs()
    dK, dKe = shared(scale * ds.transpose(-1, -2) @ q), shared(scale * (dse + F * ds.abs()).transpose(-1, -2) @ q.abs())
    dpe = p * (2.0 * dp_rel + u) + torch.where(seen, t16, 0.0)
    dV, dVe = shared(p.transpose(-1, -2) @ do), shared((dpe + F * p).transpose(-1, -2) @ do.abs())
    dQe = dQe + F * scale * ds.abs() @ kk.abs()
    val.update(dQ=dQ, dK=dK, dV=dV)
    bnd.update(dQ=dQe + u * dQ.abs() + t16, dK=dKe + u * dK.abs() + t16, dV=dVe + u * dV.abs() + t16)
    return val, bnd


def turn(x, table, positions, interleaved, inverse=False):
    """x (B,H,N,D) turned by the table rows `positions` (B,N), and its bound."""
    u = half_step(x.dtype)
    x = x.double().cpu()
    R = table.shape[1]
    row = table.double().cpu()[positions.cpu().long()][:, None]            # (B,1,N,R)
    c, s = row[..., : R // 2], row[..., R // 2:]
    if inverse:
        s = -s
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., : R // 2], x[..., R // 2: R])
    y, e = x.clone(), torch.zeros_like(x)
    first, second = a * c - b * s, b * c + a * s
    e1, e2 = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    if interleaved:
        y[..., 0:R:2], y[..., 1:R:2], e[..., 0:R:2], e[..., 1:R:2] = first, second, e1, e2
    else:
        y[..., : R // 2], y[..., R // 2: R], e[..., : R // 2], e[..., R // 2: R] = first, second, e1, e2
    out_tiny = 2.0 ** -25                                                   # fp16 below its normal range
    bound = 3 * 2.0 ** -24 * e + (u * (1 + 2.0 ** -20)) * y.abs() + out_tiny
    bound[..., R:] = 0.0
    return y, bound


def paged_dense(pages, block_row, length, page):
    """(Hkv, length, D) of one sequence, float64 on the CPU."""
    n = -(-length // page)
    x = pages.cpu()[block_row.cpu()[:n].long()].double()                    # (n, Hkv, page, D)
    return x.transpose(0, 1).flatten(1, 2)[:, :length]


def paged_attention(q, k_pages, v_pages, block_table, seq_lens, scale, softcap=0.0, slopes=None, window=0):
    """(O, lse, bound of O, bound of lse) of T new tokens a sequence."""
    dtype = q.dtype
    u, t16 = half_step(dtype), tiny(dtype)
    B, H, T, D = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    O, Oe = torch.zeros(B, H, T, D, dtype=torch.float64), torch.zeros(B, H, T, D, dtype=torch.float64)
    lse, le = torch.full((B, H, T), NEG, dtype=torch.float64), torch.zeros(B, H, T, dtype=torch.float64)
    qd = q.double().cpu()
    for b in range(B):
        n = int(seq_lens[b])
        if n == 0:
            continue
        k, v = paged_dense(k_pages, block_table[b], n, page), paged_dense(v_pages, block_table[b], n, page)
        for h in range(H):
            kh, vh = k[h * Hkv // H], v[h * Hkv // H]
            for t in range(T):
                p = n - T + t
                if p < 0:
                    continue
                first = max(0, p - window + 1) if window else 0
                x = scale * kh[first:p + 1] @ qd[b, h, t]
                e = F * (scale * kh[first:p + 1].abs() @ qd[b, h, t].abs() + 1.0)
                if softcap:
                    x = softcap * torch.tanh(x / softcap)
                    e = e + F * softcap
                if slopes is not None:
                    bias = float(slopes[h]) * torch.arange(p - first, -1, -1, dtype=torch.float64)
                    x, e = x - bias, e + F * bias
                # terms e^-40 below the largest weigh less than the roundings of the others
                near = x > x.max() - 40
                em = float(e[near].max())
                w = torch.softmax(x, -1)
                lse[b, h, t], le[b, h, t] = torch.logsumexp(x, -1), em + F * (1 + abs(float(torch.logsumexp(x, -1))))
                O[b, h, t] = w @ vh[first:p + 1]
                Oe[b, h, t] = (w * (2 * em + F + u) + t16) @ vh[first:p + 1].abs() + (u + F) * O[b, h, t].abs() + t16
    return O, lse, Oe, le


def check(got, want, bound, label=""):
    """Every element within its bound; -inf and finite places alike."""
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape, (label, got.shape, want.shape)
    finite = torch.isfinite(want)
    assert torch.equal(finite, torch.isfinite(got)), (label, "finite places differ")
    assert torch.equal(got[~finite], want[~finite]), label
    bad = (got - want).abs()[finite] - bound[finite]
    if bad.numel():
        worst = int(bad.argmax())
        assert bad.max() <= 0, (label, "off by", (got - want).abs()[finite][worst].item(), "allowed",
                                bound[finite][worst].item(), "value", want[finite][worst].item(),
                                "share outside", (bad > 0).double().mean().item())


def default_scale(D):
    return 1.0 / math.sqrt(D)
