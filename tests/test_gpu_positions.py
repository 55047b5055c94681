"""Rotary positions and the paged cache on the GPU against their 64-bit forms, element by element."""
import threading

import pytest
import torch

import exact_attention_107_b200 as fa
import operator_refs as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(autouse=True)
def _need_cuda(cuda_ok):
    yield
    assert fa.fa_device_status(reset=True) == 0


def rand(shape, dtype, seed, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(DT[dtype])


ROTARY = [
    # B, H, Hkv, N, D, R, interleaved, dtype
    (1, 1, 1, 1, 64, 64, False, "bf16"), (2, 12, 12, 1, 64, 64, True, "fp16"), (3, 4, 2, 33, 128, 128, False, "bf16"),
    (2, 5, 1, 17, 96, 96, True, "bf16"), (1, 8, 8, 65, 128, 64, True, "fp16"), (2, 3, 3, 31, 96, 50, False, "bf16"),
    (1, 2, 1, 100, 32, 8, False, "fp16"), (1, 2, 1, 100, 32, 18, True, "bf16"), (2, 4, 4, 9, 256, 256, False, "fp16"),
    (1, 40, 8, 5, 256, 64, False, "bf16"), (1, 1, 1, 200, 64, 2, False, "bf16"), (1, 1, 1, 200, 64, 2, True, "fp16"),
    (1, 2, 3, 7, 128, 66, False, "bf16"), (1, 64, 64, 3, 256, 256, True, "bf16"), (2, 7, 1, 1500, 128, 32, False, "bf16"),
]


@pytest.mark.parametrize("B,H,Hkv,N,D,R,interleaved,dtype", ROTARY)
@pytest.mark.parametrize("layout", ["contiguous", "token-major", "fused"])
def test_rotary(B, H, Hkv, N, D, R, interleaved, dtype, layout):
    rows = N + 50
    table = fa.rotary_table(rows, R, 500.0)
    g = torch.Generator().manual_seed(N)
    per_batch = torch.randint(0, rows, (B, N), generator=g, dtype=torch.int32)
    if layout == "contiguous":
        q, k = rand((B, H, N, D), dtype, 1).cuda(), rand((B, Hkv, N, D), dtype, 2).cuda()
    elif layout == "token-major":
        q, k = rand((B, N, H, D), dtype, 1).cuda().transpose(1, 2), rand((B, N, Hkv, D), dtype, 2).cuda().transpose(1, 2)
    else:                                          # one projection's output, heads side by side
        x = rand((B, N, H + 2 * Hkv, D), dtype, 3).cuda()
        q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2)
    t = table.cuda()
    for positions, flat in ((None, torch.arange(N).expand(B, N)), (per_batch, per_batch),
                            (per_batch[0], per_batch[:1].expand(B, N)), (per_batch[:1], per_batch[:1].expand(B, N))):
        pos = None if positions is None else positions.cuda()
        for call, inverse in ((fa.rotary_forward, False), (fa.rotary_backward, True)):
            got = call(q, k, t, positions=pos, interleaved=interleaved)
            for name, x, y in zip("qk", (q, k), got):
                want, bound = ref.turn(x, table, flat, interleaved, inverse)
                assert y.is_contiguous() and y.dtype == x.dtype
                ref.check(y, want, bound, (name, inverse))
    only_q, none = fa.rotary_forward(q, None, t, interleaved=interleaved)
    assert none is None
    assert torch.equal(only_q, fa.rotary_forward(q, k, t, interleaved=interleaved)[0])
    none, only_k = fa.rotary_forward(None, k, t, interleaved=interleaved)
    assert none is None
    assert torch.equal(only_k, fa.rotary_forward(q, k, t, interleaved=interleaved)[1])


def test_rotary_gradient_through_autograd():
    B, H, N, D = 2, 3, 40, 64
    table = fa.rotary_table(N, 32, scaling="by_parts", factor=4.0, original_length=16)
    q, k, gq, gk = (rand((B, H, N, D), "bf16", s).cuda() for s in range(4))
    ql, kl = q.clone().requires_grad_(), k.clone().requires_grad_()
    oq, ok = fa.rotary_embedding(ql, kl, table.cuda())
    torch.autograd.backward((oq, ok), (gq, gk))
    flat = torch.arange(N).expand(B, N)
    for leaf, grad in ((ql, gq), (kl, gk)):
        ref.check(leaf.grad, *ref.turn(grad, table, flat, False, True))
    # a gradient that arrives expanded (of a sum), one leaf of a broadcast head, one output unused
    k1 = k[:, :1].clone().requires_grad_()
    oq, ok = fa.rotary_embedding(q, k1.expand(B, H, N, D), table.cuda())
    ok.float().sum().backward()
    ones = torch.ones(B, H, N, D, dtype=torch.bfloat16)
    want, bound = ref.turn(ones, table, flat, False, True)
    u = 2.0 ** -8
    ref.check(k1.grad, want.sum(1, keepdim=True),
              bound.sum(1, keepdim=True) + H * u * (want.abs() + bound).sum(1, keepdim=True))


def test_rotary_empty_and_position_outside():
    table = fa.rotary_table(16, 64).cuda()
    q = rand((1, 2, 4, 64), "bf16", 1).cuda()
    pos = torch.tensor([3, 16, -1, 2**31 - 1], dtype=torch.int32)
    out, _ = fa.rotary_forward(q, None, table, positions=pos.cuda())
    torch.cuda.synchronize()
    assert fa.fa_device_status(reset=True) == 13
    assert torch.equal(out[:, :, 1:], q[:, :, 1:])
    want, bound = ref.turn(q[:, :, :1], table, pos[:1].expand(1, 1), False)
    ref.check(out[:, :, :1], want, bound)


# ----------------------------------------------------------------------------- paged cache
def cache(B, Hkv, D, page, longest, lens, dtype, seed):
    """Pools whose pages lie in a random order, unreached table entries -1; unused slots hold NaN."""
    g = torch.Generator().manual_seed(seed)
    wide = max(1, -(-longest // page))
    used = [-(-n // page) for n in lens]
    pool = sum(used) + 3
    order = torch.randperm(pool, generator=g).int()
    table = torch.full((B, wide), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
    k, v = rand((pool, Hkv, page, D), dtype, seed + 1), rand((pool, Hkv, page, D), dtype, seed + 2)
    free = torch.ones(pool, page, dtype=torch.bool)
    for b in range(B):
        for i in range(lens[b]):
            free[table[b, i // page], i % page] = False
    for x in (k, v):
        x.transpose(1, 2)[free] = float("nan")
    return k, v, table, free


APPEND = [
    # B, H, Hkv, T, D, R, page, interleaved, lens, new, dtype
    (1, 1, 1, 1, 64, 64, 16, False, [1], None, "bf16"),
    (3, 8, 2, 1, 128, 128, 8, False, [7, 8, 9], None, "fp16"),
    (4, 4, 4, 5, 96, 50, 16, True, [5, 40, 0, 12], [5, 1, 0, 4], "bf16"),
    (2, 5, 1, 37, 256, 256, 256, False, [300, 37], [37, 20], "bf16"),
    (3, 2, 2, 130, 32, 18, 64, False, [130, 200, 64], [130, 0, 64], "fp16"),
    (2, 6, 3, 9, 128, 32, 128, True, [9, 1000], None, "bf16"),
]


@pytest.mark.parametrize("B,H,Hkv,T,D,R,page,interleaved,lens,new,dtype", APPEND)
@pytest.mark.parametrize("with_q,with_table", [(True, True), (False, True), (False, False)])
def test_append(B, H, Hkv, T, D, R, page, interleaved, lens, new, dtype, with_q, with_table):
    table = fa.rotary_table(max(lens), R, 300.0)
    k, v, q = (rand((B, T, h, D), dtype, s).cuda().transpose(1, 2) for s, h in enumerate((Hkv, Hkv, H)))
    kp, vp, bt, _ = cache(B, Hkv, D, page, max(lens) + page, lens, dtype, 9)
    kd, vd = kp.cuda(), vp.cuda()
    q_out = fa.paged_append(k, v, kd, vd, bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                            new_lens=None if new is None else torch.tensor(new, dtype=torch.int32).cuda(),
                            q=q if with_q else None, table=table.cuda() if with_table else None, interleaved=interleaved)
    torch.cuda.synchronize()
    want_k, want_v = kp.double(), vp.double()
    bound_k = torch.zeros_like(want_k)
    for b in range(B):
        n = T if new is None else new[b]
        pos = torch.arange(lens[b] - n, lens[b])
        rows, bound = k[b:b + 1, :, :n].double().cpu(), torch.zeros(1, Hkv, n, D, dtype=torch.float64)
        if with_table and n:
            rows, bound = ref.turn(k[b:b + 1, :, :n], table, pos[None], interleaved)
        for t in range(n):
            pg, slot = int(bt[b, int(pos[t]) // page]), int(pos[t]) % page
            want_k[pg, :, slot], bound_k[pg, :, slot] = rows[0, :, t], bound[0, :, t]
            want_v[pg, :, slot] = v[b, :, t].double().cpu()
        if with_q:
            if n:
                ref.check(q_out[b:b + 1, :, :n], *ref.turn(q[b:b + 1, :, :n], table, pos[None], interleaved))
            assert (q_out[b, :, n:] == 0).all()
    assert torch.equal(torch.isnan(kd.cpu()), torch.isnan(want_k)) and torch.equal(torch.isnan(vd.cpu()), torch.isnan(want_v))
    ref.check(torch.nan_to_num(kd.cpu()), torch.nan_to_num(want_k), bound_k)
    assert torch.equal(torch.nan_to_num(vd.cpu().double()), torch.nan_to_num(want_v))


def test_append_refuses_bad_pages_on_the_device():
    """Pages outside the pool, unset pages, lengths beyond the table and new_lens beyond T or the
    length are not written; their neighbours are."""
    B, H, T, D, page = 6, 1, 2, 64, 8
    k = rand((B, H, T, D), "bf16", 1).cuda()
    kp, vp = (torch.zeros(7, H, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt = torch.tensor([[0], [7], [-1], [3], [4], [5]], dtype=torch.int32).cuda()
    lens = torch.tensor([4, 4, 4, 9, 1, 5], dtype=torch.int32).cuda()        # 9: past the table; 1: position -1
    new = torch.tensor([2, 2, 2, 2, 2, 3], dtype=torch.int32).cuda()         # 3: more than T
    fa.paged_append(k, k, kp, vp, bt, lens, new_lens=new)
    torch.cuda.synchronize()
    assert fa.fa_device_status(reset=True) == 13
    want = torch.zeros_like(kp)
    want[0, :, 2:4] = k[0]
    want[3, :, 7] = k[3, :, 0]
    want[4, :, 0] = k[4, :, 1]
    assert torch.equal(kp, want) and torch.equal(vp, want)


DECODE = [
    # B, H, Hkv, T, D, page, lens, softcap, alibi, window, dtype
    (1, 1, 1, 1, 64, 16, [1], 0.0, False, 0, "bf16"),
    (2, 12, 12, 1, 64, 16, [500, 0], 0.0, False, 0, "bf16"),
    (3, 8, 2, 1, 128, 8, [7, 8, 9], 30.0, False, 0, "fp16"),
    (4, 8, 1, 1, 128, 32, [1000, 33, 31, 513], 0.0, True, 0, "bf16"),
    (2, 5, 1, 7, 96, 64, [3, 700], 20.0, True, 0, "bf16"),
    (3, 12, 4, 5, 256, 32, [600, 128, 127], 0.0, True, 100, "fp16"),
    (2, 40, 8, 4, 128, 256, [1025, 256], 50.0, False, 1, "bf16"),
    (1, 16, 2, 1, 128, 128, [20000], 30.0, False, 0, "bf16"),
    (2, 4, 2, 64, 64, 16, [64, 900], 0.0, False, 0, "bf16"),
    (1, 64, 1, 33, 32, 8, [257], 0.0, False, 40, "fp16"),
    (5, 3, 3, 2, 32, 16, [0, 1, 2, 3, 129], 0.0, False, 0, "bf16"),
    (2, 9, 1, 3, 256, 64, [4097, 65], 0.0, False, 0, "bf16"),
    (130, 2, 1, 1, 64, 16, [n % 97 for n in range(130)], 0.0, False, 0, "fp16"),
    (1, 8, 8, 1, 96, 32, [3001], 0.0, True, 1000, "bf16"),
    # several tiles and units for each CTA, every head dim and group size
    (6, 16, 8, 1, 256, 32, [3000, 700, 2500, 0, 1500, 129], 0.0, False, 0, "bf16"),
    (6, 32, 8, 3, 256, 16, [2600, 2900, 1, 2000, 256, 1100], 0.0, True, 1000, "fp16"),
    (5, 40, 4, 3, 256, 64, [4500, 5000, 300, 3000, 2047], 30.0, False, 0, "bf16"),
    (4, 64, 8, 4, 128, 16, [4000, 2222, 3333, 90], 0.0, False, 0, "bf16"),
    (3, 64, 8, 8, 128, 32, [2000, 5000, 3500], 0.0, True, 0, "fp16"),
    (6, 16, 16, 1, 64, 8, [2000, 100, 3000, 1, 0, 1777], 0.0, False, 0, "bf16"),
    (5, 16, 16, 2, 32, 128, [2500, 128, 3000, 4000, 127], 20.0, False, 700, "fp16"),
    (4, 48, 16, 1, 96, 256, [3000, 2560, 255, 1025], 0.0, False, 0, "bf16"),
    (2, 32, 8, 13, 64, 64, [6000, 4100], 0.0, False, 0, "bf16"),
]


def decode_inputs(B, H, Hkv, T, D, page, lens, alibi, dtype):
    q = rand((B, H, T, D), dtype, 3, 2.0)
    kp, vp, bt, _ = cache(B, Hkv, D, page, max(lens) + 2 * page, lens, dtype, sum(lens) + 1)
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]) if alibi else None
    return q, kp, vp, bt, torch.tensor(lens, dtype=torch.int32), slopes


@pytest.mark.parametrize("B,H,Hkv,T,D,page,lens,cap,alibi,window,dtype", DECODE)
def test_decode(B, H, Hkv, T, D, page, lens, cap, alibi, window, dtype):
    q, kp, vp, bt, sl, slopes = decode_inputs(B, H, Hkv, T, D, page, lens, alibi, dtype)
    scale = ref.default_scale(D)
    O, lse, Oe, le = ref.paged_attention(q, kp, vp, bt, sl, scale, cap, slopes, window)
    args = [t.cuda() for t in (q, kp, vp, bt, sl)]
    more = dict(softcap=cap, alibi_slopes=None if slopes is None else slopes.cuda(), window=window)
    o, l = fa.paged_attention(*args, scale, **more)
    torch.cuda.synchronize()
    ref.check(o, O, Oe, "O")
    ref.check(l, lse, le, "lse")
    o2, l2 = fa.paged_attention(*args, scale, **more)
    assert torch.equal(o, o2) and torch.equal(l, l2)


def test_decode_bad_pages_count_as_absent():
    """A page outside the pool in the middle of a sequence, and a length beyond the table."""
    B, H, D, page = 3, 2, 64, 16
    lens = [64, 64, 64]
    q, kp, vp, bt, sl, _ = decode_inputs(B, H, H, 1, D, page, lens, False, "bf16")
    bt[0, 1], bt[1, 2] = kp.shape[0], -7
    bt = bt[:, :4].contiguous()
    sl[2] = 70
    o, lse = fa.paged_attention(*(t.cuda() for t in (q, kp, vp, bt, sl)), 0.125)
    torch.cuda.synchronize()
    assert fa.fa_device_status(reset=True) == 13
    for b, gone in ((0, 1), (1, 2), (2, None)):
        keep = [i for i in range(4) if i != gone]
        n = 16 * len(keep)
        want = ref.paged_attention(q[b:b + 1], kp, vp, bt[b:b + 1, keep], torch.tensor([n]), 0.125)
        ref.check(o[b:b + 1], want[0], want[2])
        ref.check(lse[b:b + 1], want[1], want[3])


def test_decode_two_streams_and_graphs():
    """Two calls in flight at once, and two captured graphs replayed at once, each with its own workspace."""
    cases = [decode_inputs(2, 8, 2, 1, 128, 16, [900, 5000], False, "bf16"),
             decode_inputs(3, 8, 2, 2, 128, 32, [4000, 1, 77], False, "bf16")]
    dev = [[t.cuda() for t in c[:5]] for c in cases]
    want = [fa.paged_attention(*d) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    got = [fa.paged_attention(*d, stream=s) for d, s in zip(dev, streams) for _ in range(3)]
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i // 3][0]) and torch.equal(l, want[i // 3][1])
    graphs, outs = [], []
    for d in dev:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.paged_attention(*d))
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


@pytest.mark.parametrize("dtype,D,R,interleaved,cap,alibi", [
    ("bf16", 128, 128, False, 0.0, False), ("fp16", 64, 32, True, 30.0, False), ("bf16", 96, 96, False, 0.0, True)])
def test_layer_prefilled_then_decoded(dtype, D, R, interleaved, cap, alibi):
    """One attention layer as a server runs it: the prompt through rotary_forward and attention_forward
    and into the cache, then tokens one by one and a pair through paged_append and paged_attention.
    Every step's output is the training form's row of the whole sequence."""
    B, H, Hkv, N, page = 2, 8, 2, 75, 16
    q, k, v = (rand((B, N, h, D), dtype, s, 1.5).cuda().transpose(1, 2) for s, h in enumerate((H, Hkv, Hkv)))
    table = fa.rotary_table(N, R).cuda()
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(H)]).cuda() if alibi else None
    more = dict(softcap=cap, alibi_slopes=slopes)
    qr, kr = fa.rotary_forward(q, k, table, interleaved=interleaved)
    whole, lse = fa.attention_forward(qr, kr, v.contiguous(), causal=True, **more)
    seen = ref.visible(B, N)
    want, bound = ref.attention(qr, kr, v, None, ref.default_scale(D), seen, cap, slopes)
    ref.check(whole, want["O"], bound["O"])
    kp, vp = (torch.full((2 * 5 + 1, Hkv, page, D), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
    bt = torch.randperm(11, generator=torch.Generator().manual_seed(1))[:10].view(B, 5).int().cuda()
    at = 0
    for n in (60, 1, 1, 2, 1, 9, 1):
        lens = torch.full((B,), at + n, dtype=torch.int32, device="cuda")
        part = slice(at, at + n)
        qn = fa.paged_append(k[:, :, part], v[:, :, part], kp, vp, bt, lens, q=q[:, :, part], table=table,
                             interleaved=interleaved)
        assert torch.equal(qn, qr[:, :, part])
        o, l = fa.paged_attention(qn, kp, vp, bt, lens, **more)
        ref.check(o, want["O"][:, :, part], bound["O"][:, :, part], ("O", at))
        ref.check(l, want["lse"][:, :, part], bound["lse"][:, :, part], ("lse", at))
        at += n
    assert at == N


def test_pages_before_the_window_are_not_read():
    """A server that frees the pages that slid out of the window: unset entries there are no error."""
    B, H, Hkv, T, D, page, window = 2, 8, 2, 3, 128, 16, 70
    lens = [500, 131]
    q, kp, vp, bt, sl, _ = decode_inputs(B, H, Hkv, T, D, page, lens, False, "bf16")
    want = ref.paged_attention(q, kp, vp, bt, sl, 0.1, window=window)
    for b, n in enumerate(lens):
        gone = (n - T - window + 1) // page                       # pages wholly before the first row's window
        for i in range(gone):
            kp[bt[b, i].item()], vp[bt[b, i].item()] = float("nan"), float("nan")
            bt[b, i] = -1
    o, lse = fa.paged_attention(*(t.cuda() for t in (q, kp, vp, bt, sl)), 0.1, window=window)
    torch.cuda.synchronize()
    ref.check(o, want[0], want[2])
    ref.check(lse, want[1], want[3])


def test_shared_pages_and_many_empty_sequences():
    """A common prefix in the same pages for every sequence, most of the batch empty."""
    B, H, D, page = 300, 2, 64, 16
    q, kp, vp = rand((B, H, 1, D), "bf16", 1), rand((9, H, page, D), "bf16", 2), rand((9, H, page, D), "bf16", 3)
    bt = torch.arange(9, dtype=torch.int32).repeat(B, 1)
    sl = torch.zeros(B, dtype=torch.int32)
    sl[torch.arange(3, B, 41)] = 139
    sl[299] = 1
    want = ref.paged_attention(q, kp, vp, bt, sl, 0.125)
    o, lse = fa.paged_attention(*(t.cuda() for t in (q, kp, vp, bt, sl)), 0.125)
    ref.check(o, want[0], want[2])
    ref.check(lse, want[1], want[3])


def test_largest_scores_and_equal_keys():
    """Scores of hundreds (one key takes all the weight, or all equal keys share it)."""
    B, H, D, page, n = 1, 4, 64, 16, 1000
    q, kp, vp, bt, sl, _ = decode_inputs(B, H, H, 1, D, page, [n], False, "fp16")
    for case in ("hot", "equal"):
        if case == "hot":
            q2, k2 = q * 20, kp
        else:
            q2, k2 = q, torch.where(torch.isnan(kp), kp, torch.ones_like(kp))
        for cap in (0.0, 3.0):
            want = ref.paged_attention(q2, k2, vp, bt, sl, 0.125, cap)
            o, lse = fa.paged_attention(*(t.cuda() for t in (q2, k2, vp, bt, sl)), 0.125, softcap=cap)
            ref.check(o, want[0], want[2], case)
            ref.check(lse, want[1], want[3], case)


def test_both_host_paths_agree():
    """The calls marshalled in C++ and in Python (another stream given, a workspace given)."""
    B, H, Hkv, T, D, page = 3, 8, 2, 2, 128, 16
    q, kp, vp, bt, sl, slopes = decode_inputs(B, H, Hkv, T, D, page, [100, 2, 333], True, "bf16")
    d = [t.cuda() for t in (q, kp, vp, bt, sl)]
    slopes = slopes.cuda()
    here = torch.cuda.current_stream()
    a = fa.paged_attention(*d, softcap=20.0, alibi_slopes=slopes, window=77)
    b = fa.paged_attention(*d, softcap=20.0, alibi_slopes=slopes, window=77, stream=here)
    ws = torch.empty(fa.fa_paged_workspace_size(B, H, Hkv, T, D), device="cuda", dtype=torch.uint8)
    c = fa.paged_attention(*d, softcap=20.0, alibi_slopes=slopes, window=77, workspace=ws)
    assert all(torch.equal(a[i], b[i]) and torch.equal(a[i], c[i]) for i in (0, 1))
    table = fa.rotary_table(400, 64).cuda()
    k = rand((B, T, Hkv, D), "bf16", 5).cuda().transpose(1, 2)
    pools = [[t.clone() for t in d[1:3]] for _ in range(2)]
    outs = [fa.paged_append(k, k, *p, d[3], d[4], q=d[0], table=table, stream=s) for p, s in zip(pools, (None, here))]
    assert torch.equal(*outs) and all(torch.equal(torch.nan_to_num(x), torch.nan_to_num(y)) for x, y in zip(*pools))
    x, y = fa.rotary_forward(d[0], k, table), fa.rotary_forward(d[0], k, table, stream=here)
    assert all(torch.equal(i, j) for i, j in zip(x, y))


def test_refusals_with_gpu_tensors():
    """What the C++ path hands back is refused by the Python path, with its messages."""
    B, H, D, page = 1, 2, 64, 16
    q, kp, vp, bt, sl, _ = decode_inputs(B, H, H, 1, D, page, [20], False, "bf16")
    q, kp, vp, bt, sl = (t.cuda() for t in (q, kp, vp, bt, sl))
    table = fa.rotary_table(40, 64).cuda()
    odd = torch.zeros(1, 2, 1, 72, device="cuda", dtype=torch.bfloat16)[..., 4:68]
    for error, call in [
        (TypeError, lambda: fa.rotary_forward(q.float(), q.float(), table)),
        (ValueError, lambda: fa.rotary_forward(odd, q, table)),
        (ValueError, lambda: fa.rotary_forward(q, q[..., :32].contiguous(), table)),
        (ValueError, lambda: fa.rotary_forward(q, q, table[:, :63].contiguous())),
        (ValueError, lambda: fa.rotary_forward(q, q, table[:, :32])),
        (TypeError, lambda: fa.rotary_forward(q, q, table.half())),
        (TypeError, lambda: fa.rotary_forward(q, q, table, positions=torch.zeros(1, 1, device="cuda", dtype=torch.int64))),
        (ValueError, lambda: fa.rotary_forward(q, q, table, positions=torch.zeros(2, 1, device="cuda", dtype=torch.int32))),
        (ValueError, lambda: fa.rotary_forward(q, q, fa.rotary_table(4, 66).cuda())),
        (TypeError, lambda: fa.paged_append(q, q, kp.half(), vp, bt, sl)),
        (ValueError, lambda: fa.paged_append(q, q[:, :1], kp, vp, bt, sl)),
        (ValueError, lambda: fa.paged_append(q, q, kp, vp[:, :1].contiguous(), bt, sl)),
        (ValueError, lambda: fa.paged_append(q, q, kp, vp, bt[0], sl)),
        (TypeError, lambda: fa.paged_append(q, q, kp, vp, bt.long(), sl)),
        (ValueError, lambda: fa.paged_append(q, q, kp, vp, bt, sl, q=q)),
        (fa.FAError, lambda: fa.paged_append(q, q, kp[:, :, :12].contiguous(), vp[:, :, :12].contiguous(), bt, sl)),
        (ValueError, lambda: fa.paged_attention(q, kp, vp, bt, sl[None])),
        (ValueError, lambda: fa.paged_attention(q.expand(2, 2, 1, 64), kp, vp, bt, sl)),
        (TypeError, lambda: fa.paged_attention(q, kp, vp.float(), bt, sl)),
        (fa.FAError, lambda: fa.paged_attention(q, kp, vp, bt, sl, -1.0)),
        (fa.FAError, lambda: fa.paged_attention(q, kp, vp, bt, sl, window=-2)),
        (fa.FAError, lambda: fa.paged_attention(q[:, :, :0].contiguous(), kp, vp, bt, sl)),
        (fa.FAError, lambda: fa.paged_attention(q.expand(1, 2, 65, 64).contiguous(), kp, vp, bt, sl)),
        (fa.FAError, lambda: fa.paged_attention(q, kp, vp, bt, sl, workspace=torch.empty(16, device="cuda", dtype=torch.uint8))),
        (ValueError, lambda: fa.paged_attention(q, kp, vp, bt, sl, alibi_slopes=torch.ones(3, device="cuda"))),
    ]:
        with pytest.raises(error):
            call()


def test_pool_beyond_32_bit_offsets():
    """Pages behind the 2^31st element of a pool, appended to and read back."""
    B, H, Hkv, T, D, page, pages = 2, 16, 8, 40, 128, 256, 8300
    assert pages * Hkv * page * D > 2 ** 31
    kp, vp = (torch.empty(pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt = torch.tensor([[pages - 1, 0, pages - 3], [7, pages - 2, -1]], dtype=torch.int32)
    q, k, v = (rand((B, 600, h, D), "bf16", s) for s, h in enumerate((H, Hkv, Hkv)))
    lens = [600, 300]
    cu = lambda t, a, b: t[:, a:b].contiguous().cuda().transpose(1, 2)
    for a in range(0, 600, T):                                    # position p of sequence b holds row p
        new = torch.tensor([max(0, min(T, n - a)) for n in lens], dtype=torch.int32).cuda()
        at = torch.tensor([min(n, a + T) for n in lens], dtype=torch.int32).cuda()
        fa.paged_append(cu(k, a, a + T), cu(v, a, a + T), kp, vp, bt.cuda(), at, new_lens=new)
    sl = torch.tensor(lens, dtype=torch.int32)
    q1 = q[:, :1].transpose(1, 2).contiguous()
    o, lse = fa.paged_attention(q1.cuda(), kp, vp, bt.cuda(), sl.cuda())
    small_k, small_v = (torch.zeros(6, Hkv, page, D, dtype=torch.bfloat16) for _ in range(2))
    small = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32)
    for b, n in enumerate(lens):
        for p in range(n):
            small_k[small[b, p // page], :, p % page], small_v[small[b, p // page], :, p % page] = k[b, p], v[b, p]
    want = ref.paged_attention(q1, small_k, small_v, small, sl, ref.default_scale(D))
    ref.check(o, want[0], want[2])
    ref.check(lse, want[1], want[3])


def test_rotary_embedding_of_one_tensor():
    """Only q or only k, their gradients, and a second backward through them refused."""
    table = fa.rotary_table(30, 64).cuda()
    x = rand((2, 2, 30, 64), "bf16", 4).cuda().requires_grad_()
    flat = torch.arange(30).expand(2, 30)
    for args in ((x, None), (None, x)):
        out = [t for t in fa.rotary_embedding(*args, table) if t is not None]
        assert len(out) == 1
        g = rand((2, 2, 30, 64), "bf16", 5).cuda()
        grad, = torch.autograd.grad(out[0], x, g, create_graph=True)
        ref.check(grad.detach(), *ref.turn(g, table, flat, False, True))
        with pytest.raises(RuntimeError):
            grad.float().sum().backward()


def test_calls_from_several_threads():
    """Eight threads, each on its own stream, at once: every result is the single call's."""
    B, H, Hkv, T, D, page = 2, 8, 2, 1, 64, 16
    q, kp, vp, bt, sl, _ = decode_inputs(B, H, Hkv, T, D, page, [700, 90], False, "bf16")
    d = [t.cuda() for t in (q, kp, vp, bt, sl)]
    x, table = rand((2, 3, 50, 64), "bf16", 2).cuda(), fa.rotary_table(50, 64).cuda()
    want = fa.paged_attention(*d) + (fa.rotary_forward(x, None, table)[0],)
    torch.cuda.synchronize()
    bad = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                got = fa.paged_attention(*d) + (fa.rotary_forward(x, None, table)[0],)
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                bad.append(1)
            stream.synchronize()

    threads = [threading.Thread(target=work) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
