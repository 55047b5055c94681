"""Cases, plain forms and 64-bit definitions of the operators around the attention call:

    rotary     rotary positions of queries and keys, forward and backward
    append     new keys and values written into a paged cache, rotated on the way with the queries
    decode     attention of one or a few new tokens over a paged cache
    attention  attention with capped scores, a distance bias, document / prefix / window masks and
               shared key-value heads, forward alone or with its gradients

run() computes the plain form with elementary torch operations in 32 bits, or, where `own` is set,
calls the framework's entry points.  The batch's lengths and documents follow from the case alone,
the values from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
NEG = float("-inf")


def _package():
    import exact_attention_107_b200 as fa
    return fa


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of a small model: a handful of rows, all latency.
        dict(name="rotary forward, one token", op="rotary", direction="forward", B=4, H=12, Hkv=12, N=1, D=64, R=64,
             interleaved=False, packed=True, dtype="bf16"),
        # Training step, queries and keys straight from the projections (token-major views), whole heads, half layout.
        dict(name="rotary forward, training", op="rotary", direction="forward", B=8, H=16, Hkv=4, N=4096, D=128,
             R=128, interleaved=False, packed=False, dtype="bf16"),
        # Its gradient where only part of the head turns, interleaved pairs, packed documents.
        dict(name="rotary backward, part of the head", op="rotary", direction="backward", B=1, H=8, Hkv=8, N=32767,
             D=128, R=64, interleaved=True, packed=True, dtype="fp16"),
        # One decode step of a full batch: each sequence writes one token somewhere in its last page.
        dict(name="append, one token of 64 sequences", op="append", B=64, H=32, Hkv=8, T=1, D=128, R=128, page=16,
             interleaved=False, longest=4096, ragged=False, dtype="bf16"),
        # Prompt rows of unequal lengths enter the cache.
        dict(name="append, ragged prompts", op="append", B=5, H=16, Hkv=4, T=2000, D=128, R=96, page=64,
             interleaved=True, longest=4096, ragged=True, dtype="fp16"),
        # One sequence, short cache: latency.
        dict(name="decode, one short sequence", op="decode", B=1, H=12, Hkv=12, T=1, D=64, page=16, longest=500,
             softcap=0.0, alibi=False, window=0, dtype="bf16"),
        # A serving batch of unequal lengths with shared heads, small pages.
        dict(name="decode, ragged batch of 48", op="decode", B=48, H=32, Hkv=8, T=1, D=128, page=16, longest=8192,
             softcap=0.0, alibi=False, window=0, dtype="bf16"),
        # One very long cache: all the parallelism has to come from splitting its length.
        dict(name="decode, one long sequence", op="decode", B=1, H=16, Hkv=2, T=1, D=128, page=128, longest=262144,
             softcap=30.0, alibi=False, window=0, dtype="bf16"),
        # A few drafted tokens a sequence, wide heads, distance bias and a window.
        dict(name="decode, drafted tokens in a window", op="decode", B=17, H=12, Hkv=4, T=5, D=256, page=32,
             longest=6000, softcap=0.0, alibi=True, window=4096, dtype="fp16"),
        # A training step of a short causal model with a distance bias.
        dict(name="attention step, distance bias", op="attention", direction="both", B=8, H=12, Hkv=12, N=1024, D=64,
             mask="causal", softcap=0.0, alibi=True, dtype="bf16"),
        # A prefix mask on an odd length, forward alone.
        dict(name="attention forward, prefix", op="attention", direction="forward", B=2, H=16, Hkv=2, N=2777, D=96,
             mask="prefix", softcap=50.0, alibi=False, dtype="fp16"),
        # A packed long training step: documents of many lengths, capped scores, shared heads.
        dict(name="attention step, packed documents", op="attention", direction="both", B=1, H=8, Hkv=2, N=16384,
             D=128, mask="documents", softcap=30.0, alibi=False, dtype="bf16"),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "decode", "attention", "decode", "attention"])
    dtype = rng.choice(["bf16", "fp16"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 1, 2, 4, 5, 8])
    if op in ("rotary", "append"):
        D = rng.choice([32, 64, 96, 128, 256])
        R = rng.choice([D, D, D // 2, D // 4, D // 2 + 2])
        case = dict(op=op, B=_log(rng, 1, 64), H=Hkv * group, Hkv=Hkv, D=D, R=R, interleaved=rng.random() < 0.5,
                    dtype=dtype)
        most = 48_000_000 // (case["B"] * (case["H"] + case["Hkv"]) * D)      # elements of one call
        if op == "rotary":
            return dict(case, direction=rng.choice(["forward", "backward"]), N=_log(rng, 1, max(1, min(32768, most))),
                        packed=rng.random() < 0.5)
        T = _log(rng, 1, max(1, min(2048, most)))
        longest = T + _log(rng, 1, 4096)
        while case["B"] * longest * Hkv * D > 160_000_000:
            case["B"] = max(1, case["B"] // 2)
        return dict(case, T=T, page=rng.choice([8, 16, 32, 64, 128, 256]), longest=longest, ragged=rng.random() < 0.5)
    softcap = rng.choice([0.0, 0.0, 20.0, 30.0, 50.0])
    if op == "decode":
        D = rng.choice([32, 64, 96, 128, 256])
        B = _log(rng, 1, 128)
        longest = _log(rng, 1, max(16, min(131072, 400_000_000 // (B * Hkv * D))))
        return dict(op=op, B=B, H=Hkv * group, Hkv=Hkv, T=rng.choice([1, 1, 1, 2, 4, 7]), D=D,
                    page=rng.choice([8, 16, 32, 64, 128, 256]), longest=longest, softcap=softcap,
                    alibi=rng.random() < 0.3, window=rng.choice([0, 0, 0, _log(rng, 1, longest)]), dtype=dtype)
    B, D = rng.choice([1, 1, 2, 3, 4]), rng.choice([32, 64, 96, 128])
    H = Hkv * group
    direction = rng.choice(["forward", "both", "both"])
    N = _log(rng, 1 if direction == "forward" else 40, 8192)     # gradients of a single key are zero
    while B * H * N * N * D > 8 * 16384 * 16384 * 128 // 10:
        N = N * 3 // 4
    return dict(op=op, direction=direction, B=B, H=H, Hkv=Hkv, N=N, D=D,
                mask=rng.choice(["full", "causal", "documents", "documents full", "prefix", "window"]),
                softcap=softcap, alibi=rng.random() < 0.3, dtype=dtype)


# ----------------------------------------------------------------------------- what follows from the case alone
def _rand(case):
    text = ",".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name")
    return np.random.RandomState(sum((i + 1) * ord(c) for i, c in enumerate(text)) % (1 << 31))


def _lengths(case):
    """Cache lengths of a decode or append batch: one sequence of the longest length, the others spread from
    nothing up to it (an appended row count is at most the length)."""
    r, B, most = _rand(case), case["B"], case["longest"]
    lens = np.minimum(most, (most * r.uniform(0.0, 1.2, B)).astype(np.int64))
    lens[r.randint(B)] = most
    if case["op"] == "append":
        new = np.full(B, case["T"], np.int64)
        if case["ragged"]:
            new = np.minimum(case["T"], (case["T"] * r.uniform(0.0, 1.3, B)).astype(np.int64))
            new[r.randint(B)] = case["T"]
        return np.maximum(lens, new), new
    return lens, None


def _documents(case):
    """(B, N) document ids: lengths spread over a factor of 16 around N / 6, a padded tail (-1) in every second
    batch row."""
    r, B, N = _rand(case), case["B"], case["N"]
    ids = np.zeros((B, N), np.int32)
    for b in range(B):
        at, n = 0, 0
        while at < N:
            size = max(1, int(N / 6 * 4 ** r.uniform(-1, 1)))
            ids[b, at:at + size] = n
            at, n = at + size, n + 1
        if b % 2 == 1 or (B == 1 and N > 64):
            ids[b, N - N // 50:] = -1
    return ids


def _prefixes(case):
    r = _rand(case)
    return r.randint(0, case["N"] + 1, case["B"]).astype(np.int32)


def _window(case):
    return max(1, case["N"] // 5)


def _intervals(case):
    """(B, N) first and one-past-last visible key of each row."""
    B, N = case["B"], case["N"]
    i = np.broadcast_to(np.arange(N), (B, N))
    lo, hi = np.zeros((B, N), np.int64), np.full((B, N), N)
    kind = case["mask"]
    if kind.startswith("documents"):
        ids = _documents(case)
        for b in range(B):
            edge = np.flatnonzero(np.diff(ids[b])) + 1
            first, last = np.concatenate([[0], edge]), np.concatenate([edge, [N]])
            lo[b], hi[b] = np.repeat(first, last - first), np.repeat(last, last - first)
        hi = np.where(ids < 0, lo, hi)
    if kind in ("causal", "documents", "window"):
        hi = np.minimum(hi, i + 1)
    if kind == "prefix":
        hi = np.maximum(i + 1, _prefixes(case)[:, None])
    if kind == "window":
        lo = np.maximum(lo, i + 1 - _window(case))
    return lo, np.maximum(hi, lo)


def _span(case, length):
    """Cached positions that a decode step of one sequence has to read."""
    start = max(0, length - case["T"] + 1 - case["window"]) if case["window"] else 0
    return max(0, length - min(start, length))


def work(case):
    op, D, H, Hkv = case["op"], case["D"], case["H"], case["Hkv"]
    if op == "rotary":
        n = case["B"] * case["N"]
        table = 4 * case["R"] * (n if case["packed"] else case["N"])
        return {"bytes": 4 * n * (H + Hkv) * D + table, "flops": 3 * n * (H + Hkv) * case["R"]}
    if op == "append":
        lens, new = _lengths(case)
        n, rows = int(new.sum()), case["B"] * case["T"]
        return {"bytes": 2 * (n * (H + 4 * Hkv) + rows * H) * D + 4 * case["R"] * n, "flops": 3 * n * (H + Hkv) * case["R"]}
    if op == "decode":
        lens, _ = _lengths(case)
        read = sum(_span(case, int(n)) for n in lens)
        rows = case["B"] * H * case["T"]
        return {"bytes": 4 * read * Hkv * D + 4 * rows * D + 4 * rows, "flops": 4 * read * H * case["T"] * D}
    lo, hi = _intervals(case)
    pairs = int((hi - lo).sum()) * H
    rows, shared = case["B"] * H * case["N"], case["B"] * Hkv * case["N"]
    if case["direction"] == "forward":
        return {"bytes": 4 * rows * D + 4 * shared * D + 4 * rows, "flops": 4 * pairs * D}
    return {"bytes": 8 * rows * D + 8 * shared * D + 4 * rows, "flops": 14 * pairs * D}


# ----------------------------------------------------------------------------- inputs
def _table(positions, R, device):
    """cos | sin of position * frequency, from 64-bit angles; frequencies stretched fourfold for a long context."""
    freq = 10000.0 ** (-torch.arange(0, R, 2, device=device, dtype=torch.float64) / R) / 4.0
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _slopes(H, device):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device=device)


def _pages(case, lens, new_normal, g, device):
    """A pool of pages and the block table of a batch whose pages lie in it in a random order; entries that no
    sequence has reached yet are -1."""
    B, page = case["B"], case["page"]
    wide = -(-case["longest"] // page)
    used = (lens + page - 1) // page
    pool = int(used.sum()) + 3
    order = torch.randperm(pool, generator=g, device=device).to(torch.int32)
    table = torch.full((B, wide), -1, dtype=torch.int32, device=device)
    at = torch.from_numpy(np.arange(wide)[None, :] < used[:, None]).to(device)
    table[at] = order[: int(used.sum())]
    k, v = (new_normal(pool, case["Hkv"], page, case["D"]) for _ in range(2))
    return k, v, table


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dtype)

    s = {"case": case}
    op, B, H, Hkv, D = case["op"], case["B"], case["H"], case["Hkv"], case["D"]
    if op == "rotary":
        N = case["N"]
        s["table"] = _table(N + 4096, case["R"], dev)
        s["positions"] = None
        if case["packed"]:                                   # documents that begin anew, or caches of some length
            start = torch.randint(0, 4096, (B, 1), generator=g, device=dev)
            s["positions"] = ((torch.arange(N, device=dev)[None] + start) % (N + 4096)).to(torch.int32)
        if case["direction"] == "forward":                   # token-major views, as the projections give them
            s["q"], s["k"] = normal(B, N, H, D).transpose(1, 2), normal(B, N, Hkv, D).transpose(1, 2)
        else:
            s["q"], s["k"] = normal(B, H, N, D), normal(B, Hkv, N, D)
    elif op == "append":
        T = case["T"]
        lens, new = _lengths(case)
        s["k_pages"], s["v_pages"], s["block_table"] = _pages(case, lens, normal, g, dev)
        s["seq_lens"] = torch.from_numpy(lens.astype(np.int32)).to(dev)
        s["new_lens"] = torch.from_numpy(new.astype(np.int32)).to(dev) if case["ragged"] else None
        s["table"] = _table(case["longest"], case["R"], dev)
        s["q"], s["k"], s["v"] = (normal(B, T, h, D).transpose(1, 2) for h in (H, Hkv, Hkv))
    elif op == "decode":
        lens, _ = _lengths(case)
        s["k_pages"], s["v_pages"], s["block_table"] = _pages(case, lens, normal, g, dev)
        s["seq_lens"] = torch.from_numpy(lens.astype(np.int32)).to(dev)
        s["q"] = normal(B, H, case["T"], D, std=2.0)
        s["slopes"] = _slopes(H, dev) if case["alibi"] else None
    else:
        N = case["N"]
        s["q"], s["k"], s["v"] = normal(B, H, N, D, std=2.0), normal(B, Hkv, N, D), normal(B, Hkv, N, D)
        s["do"] = normal(B, H, N, D) if case["direction"] == "both" else None
        s["slopes"] = _slopes(H, dev) if case["alibi"] else None
        kind = case["mask"]
        s["documents"] = torch.from_numpy(_documents(case)).to(dev) if kind.startswith("documents") else None
        s["prefix"] = torch.from_numpy(_prefixes(case)).to(dev) if kind == "prefix" else None
    return s


# ----------------------------------------------------------------------------- one pass
def run(s):
    return {"rotary": _rotary, "append": _append, "decode": _decode, "attention": _attention}[s["case"]["op"]](s)


def _turn(x, cos, sin, R, interleaved):
    """The pairs of the first R columns of x (float) turned by the angles whose cos and sin are given."""
    turned, rest = x[..., :R], x[..., R:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        out = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turned[..., : R // 2], turned[..., R // 2:]
        out = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([out, rest], -1)


def _rotary(s):
    case, q, k = s["case"], s["q"], s["k"]
    forward = case["direction"] == "forward"
    if own:
        call = _package().rotary_forward if forward else _package().rotary_backward
        return call(q, k, s["table"], positions=s["positions"], interleaved=case["interleaved"])
    R, N = case["R"], case["N"]
    at = s["table"][:N][None] if s["positions"] is None else s["table"][s["positions"].long()]
    cos, sin = at[:, None, :, : R // 2], at[:, None, :, R // 2:]
    sin = sin if forward else -sin
    return tuple(_turn(x.float(), cos, sin, R, case["interleaved"]).to(x.dtype) for x in (q, k))


def _append(s):
    case = s["case"]
    if own:
        q = _package().paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"],
                                    new_lens=s["new_lens"], q=s["q"], table=s["table"],
                                    interleaved=case["interleaved"])
        return q, s["k_pages"], s["v_pages"]
    T, R, page, dev = case["T"], case["R"], case["page"], s["q"].device
    t = torch.arange(T, device=dev)
    new = torch.full_like(s["seq_lens"], T) if s["new_lens"] is None else s["new_lens"]
    real = t[None] < new[:, None]
    at = torch.where(real, (s["seq_lens"] - new)[:, None] + t[None], 0).long()
    angles = s["table"][at][:, None]
    cos, sin = angles[..., : R // 2], angles[..., R // 2:]
    q = torch.where(real[:, None, :, None], _turn(s["q"].float(), cos, sin, R, case["interleaved"]), 0.0).to(s["q"].dtype)
    k = _turn(s["k"].float(), cos, sin, R, case["interleaved"]).to(s["k"].dtype)
    b, tt = real.nonzero(as_tuple=True)
    p = at[b, tt]
    where = s["block_table"][b, p // page].long()
    s["k_pages"][where, :, p % page] = k[b, :, tt]
    s["v_pages"][where, :, p % page] = s["v"][b, :, tt]
    return q, s["k_pages"], s["v_pages"]


def _dense(pages, table):
    """(B, Hkv, positions, D): the pages of each sequence one behind the other."""
    x = pages[table.clamp(min=0).long()]                     # (B, wide, Hkv, page, D)
    return x.transpose(1, 2).flatten(2, 3)


def _softmax(x, visible):
    """Row-wise softmax of x over the visible places and the logarithm of its sum; rows that see nothing give zeros."""
    x = torch.where(visible, x, NEG)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG, 0.0, m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    return p, (m + torch.log(total)).squeeze(-1)


def _decode(s):
    case = s["case"]
    scale = case["D"] ** -0.5
    if own:
        return _package().paged_attention(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], scale,
                                          softcap=case["softcap"], alibi_slopes=s["slopes"], window=case["window"])
    B, H, Hkv, T, D = (case[n] for n in ("B", "H", "Hkv", "T", "D"))
    k, v = _dense(s["k_pages"], s["block_table"]), _dense(s["v_pages"], s["block_table"])
    L, dev = k.shape[2], k.device
    j = torch.arange(L, device=dev)
    p = s["seq_lens"][:, None].long() - T + torch.arange(T, device=dev)[None]              # (B, T)
    visible = j <= p[..., None]
    if case["window"]:
        visible &= j > p[..., None] - case["window"]
    visible = visible[:, None, None]                                                       # (B, 1, 1, T, L)
    q = s["q"].float().view(B, Hkv, H // Hkv * T, D)
    x = (q @ k.float().transpose(-1, -2)).view(B, Hkv, H // Hkv, T, L) * scale
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    if s["slopes"] is not None:
        x = x - s["slopes"].view(Hkv, -1, 1, 1) * (p[:, None, None, :, None] - j).abs().float()
    w, lse = _softmax(x, visible)
    v = torch.where((j < s["seq_lens"][:, None])[:, None, :, None], v.float(), 0.0)
    o = w.view(B, Hkv, -1, L) @ v
    return o.view(B, H, T, D).to(s["q"].dtype), lse.reshape(B, H, T)


def _visible(s):
    """(B or 1, 1, N, N): which keys a row may see."""
    case = s["case"]
    kind, N = case["mask"], case["N"]
    i = torch.arange(N, device=s["q"].device)
    near = i[None, :] <= i[:, None] if kind in ("causal", "documents", "window", "prefix") else i[None, :] >= 0
    near = near.expand(1, N, N)
    if kind.startswith("documents"):
        ids = s["documents"]
        near = near & (ids[:, :, None] == ids[:, None, :]) & (ids >= 0)[:, :, None]
    if kind == "prefix":
        near = near | (i[None, None, :] < s["prefix"][:, None, None])
    if kind == "window":
        near = near & (i[None, :] > i[:, None] - _window(case))
    return near[:, None]


def _attention(s):
    case = s["case"]
    B, H, Hkv, N, D = (case[n] for n in ("B", "H", "Hkv", "N", "D"))
    scale, cap, kind, slopes = D ** -0.5, case["softcap"], case["mask"], s["slopes"]
    q, k, v, do = s["q"], s["k"], s["v"], s["do"]
    if own:
        fa = _package()
        mask = None
        if kind not in ("causal", "full"):
            mask = fa.attention_mask(B, N, documents=s["documents"], prefix=s["prefix"], causal=kind != "documents full",
                                     window=_window(case) if kind == "window" else 0, device=q.device)
        more = dict(mask=mask, softcap=cap, alibi_slopes=slopes)
        o, lse = fa.attention_forward(q, k, v, scale, kind == "causal", **more)
        if do is None:
            return o, lse
        return (o, lse) + fa.attention_backward(q, k, v, o, lse, do, scale, kind == "causal", **more)
    G = H // Hkv
    qf = q.float().view(B, Hkv, G * N, D)
    kf, vf = k.float(), v.float()
    x = (qf @ kf.transpose(-1, -2)).view(B, H, N, N).mul_(scale)
    bend = None
    if cap:
        bend = torch.tanh(x.div_(cap))
        x = cap * bend
    if slopes is not None:
        i = torch.arange(N, device=q.device)
        x = x - slopes[:, None, None] * (i[:, None] - i[None, :]).abs().float()
    p, lse = _softmax(x, _visible(s))
    del x
    o = (p.view(B, Hkv, G * N, N) @ vf).view(B, H, N, D)
    if do is None:
        return o.to(q.dtype), lse
    dof = do.float().view(B, Hkv, G * N, D)
    dv = p.view(B, Hkv, G * N, N).transpose(-1, -2) @ dof
    ds = (dof @ vf.transpose(-1, -2)).view(B, H, N, N)
    ds = ds.sub_((do.float() * o).sum(-1, keepdim=True)).mul_(p)
    if cap:
        ds = ds.mul_(1.0 - bend.square_())
    ds = ds.view(B, Hkv, G * N, N)
    dq = (ds @ kf).view(B, H, N, D) * scale
    dk = ds.transpose(-1, -2) @ qf * scale
    return tuple(t.to(q.dtype) if t is not lse else t for t in (o, lse, dq, dk, dv))


# ----------------------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "append": _exact_append, "decode": _exact_decode,
            "attention": _exact_attention}[case["op"]](s)


def _complex_turn(x, angles, R, interleaved, inverse=False):
    """Pairs as complex numbers times cos + i sin."""
    x = x.double()
    w = torch.complex(angles[..., : R // 2].double(), angles[..., R // 2:].double())
    if inverse:
        w = w.conj()
    out = x.clone()
    if interleaved:
        z = torch.view_as_complex(x[..., :R].reshape(*x.shape[:-1], R // 2, 2).contiguous()) * w
        out[..., :R] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., : R // 2].contiguous(), x[..., R // 2: R].contiguous()) * w
        out[..., : R // 2], out[..., R // 2: R] = z.real, z.imag
    return out


def _exact_rotary(s):
    case = s["case"]
    B, N = case["B"], case["N"]
    at = torch.arange(N, device=s["q"].device).expand(B, N) if s["positions"] is None else s["positions"].long()
    inverse = case["direction"] == "backward"
    return tuple(torch.stack([_complex_turn(x[b], s["table"][at[b]], case["R"], case["interleaved"], inverse)
                              for b in range(B)]) for x in (s["q"], s["k"]))


def _exact_append(s):
    case = s["case"]
    T, page = case["T"], case["page"]
    lens = s["seq_lens"].tolist()
    new = [T] * case["B"] if s["new_lens"] is None else s["new_lens"].tolist()
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    for b in range(case["B"]):
        n, first = new[b], lens[b] - new[b]
        if n == 0:
            continue
        angles = s["table"][first:first + n]
        q[b, :, :n] = _complex_turn(s["q"][b, :, :n], angles, case["R"], case["interleaved"])
        k = _complex_turn(s["k"][b, :, :n], angles, case["R"], case["interleaved"])
        p = torch.arange(first, first + n, device=q.device)
        ids = s["block_table"][b].long()[p // page]
        kp[ids, :, p % page] = k.transpose(0, 1)
        vp[ids, :, p % page] = s["v"][b, :, :n].double().transpose(0, 1)
    return q, kp, vp


def _exact_decode(s):
    case = s["case"]
    B, H, Hkv, T, D, page = (case[n] for n in ("B", "H", "Hkv", "T", "D", "page"))
    dev = s["q"].device
    o = torch.zeros(B, H, T, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, H, T), NEG, dtype=torch.float64, device=dev)
    for b, n in enumerate(s["seq_lens"].tolist()):
        if n == 0:
            continue
        ids = s["block_table"][b, : -(-n // page)].long()
        for h in range(Hkv):
            k, v = (x[ids, h].double().reshape(-1, D)[:n] for x in (s["k_pages"], s["v_pages"]))
            for t in range(T):
                p = n - T + t
                first = max(0, p - case["window"] + 1) if case["window"] else 0
                if p < 0:
                    continue
                heads = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
                x = s["q"][b, heads, t].double() @ k[first:p + 1].T / math.sqrt(D)
                if case["softcap"]:
                    x = torch.tanh(x / case["softcap"]) * case["softcap"]
                if s["slopes"] is not None:
                    x = x - s["slopes"][heads, None].double() * torch.arange(p - first, -1, -1, device=dev)
                lse[b, heads, t] = torch.logsumexp(x, -1)
                o[b, heads, t] = torch.softmax(x, -1) @ v[first:p + 1]
    return o, lse


def _exact_attention(s):
    """Head by head, a block of rows at a time, over each row's interval of keys."""
    case = s["case"]
    B, H, Hkv, N, D = (case[n] for n in ("B", "H", "Hkv", "N", "D"))
    dev, cap, scale = s["q"].device, case["softcap"], 1.0 / math.sqrt(D)
    lo, hi = (torch.from_numpy(np.ascontiguousarray(x)).to(dev) for x in _intervals(case))
    j = torch.arange(N, device=dev)
    f64 = dict(dtype=torch.float64, device=dev)
    o, lse, dq = torch.zeros(B, H, N, D, **f64), torch.zeros(B, H, N, **f64), torch.zeros(B, H, N, D, **f64)
    dk, dv = torch.zeros(B, Hkv, N, D, **f64), torch.zeros(B, Hkv, N, D, **f64)
    for b in range(B):
        for h in range(H):
            n = h * Hkv // H
            k, v = s["k"][b, n].double(), s["v"][b, n].double()
            for r in range(0, N, 4096):
                rows = slice(r, min(N, r + 4096))
                q = s["q"][b, h, rows].double()
                x = scale * (q @ k.T)
                slope = 1.0
                if cap:
                    t = torch.tanh(x / cap)
                    x, slope = cap * t, 1.0 - t * t
                if s["slopes"] is not None:
                    x = x - s["slopes"][h].double() * (j[rows, None] - j).abs()
                x = x.masked_fill((j < lo[b, rows, None]) | (j >= hi[b, rows, None]), NEG)
                sums = torch.logsumexp(x, -1)
                p = torch.exp(x - torch.where(sums == NEG, 0.0, sums)[:, None])
                lse[b, h, rows], o[b, h, rows] = sums, p @ v
                if s["do"] is None:
                    continue
                do = s["do"][b, h, rows].double()
                dv[b, n] += p.T @ do
                dp = do @ v.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * slope
                dq[b, h, rows] = scale * (ds @ k)
                dk[b, n] += scale * (ds.T @ q)
    return (o, lse) if s["do"] is None else (o, lse, dq, dk, dv)
