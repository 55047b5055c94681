"""Edges of the rotary, paged-cache and score-modified operators on the GPU: what lies outside a
table, masked rows of the largest values, single keys, sizes beyond C's integers, both host paths."""
import pytest
import torch

import exact_attention_107_b200 as fa
import exact_attention_107_b200._binding as base
import operator_refs as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(autouse=True)
def _need_cuda(cuda_ok):
    yield
    assert fa.fa_device_status(reset=True) == 0


def rand(shape, dtype, seed, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(DT[dtype])


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("R,interleaved", [(64, False), (32, False), (34, False), (64, True), (18, True)])
def test_append_leaves_out_positions_past_the_rotary_table(R, interleaved):
    """A key whose angles the table does not hold is not written, nor its value; q's row stays unturned."""
    B, H, Hkv, T, D, page, rows = 3, 3, 2, 3, 64, 16, 20
    lens = [20, 22, 25]                                  # positions 17-19, 19-21, 22-24
    table = fa.rotary_table(rows, R)
    q, k, v = (rand((B, h, T, D), "bf16", s) for s, h in enumerate((H, Hkv, Hkv)))
    kp, vp = (torch.zeros(2 * B, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt = torch.arange(2 * B, dtype=torch.int32).view(B, 2)
    out = fa.paged_append(k.cuda(), v.cuda(), kp, vp, bt.cuda(), ints(*lens).cuda(), q=q.cuda(), table=table.cuda(),
                          interleaved=interleaved)
    torch.cuda.synchronize()
    assert fa.fa_device_status(reset=True) == 13
    want_k, want_v, bound = (torch.zeros(kp.shape, dtype=torch.float64) for _ in range(3))
    for b in range(B):
        for t in range(T):
            p = lens[b] - T + t
            one = slice(b, b + 1), slice(None), slice(t, t + 1)
            if p >= rows:
                assert torch.equal(out[one].cpu(), q[one])
                continue
            ref.check(out[one], *ref.turn(q[one], table, torch.tensor([[p]]), interleaved))
            at = int(bt[b, p // page]), slice(None), p % page
            y, e = ref.turn(k[one], table, torch.tensor([[p]]), interleaved)
            want_k[at], bound[at], want_v[at] = y[0, :, 0], e[0, :, 0], v[b, :, t].double()
    ref.check(kp, want_k, bound)
    assert torch.equal(vp.cpu().double(), want_v)


@pytest.mark.parametrize("D,page,T", [(64, 16, 2), (128, 16, 1), (128, 128, 3), (256, 32, 2)])
def test_capped_decode_does_not_depend_on_unused_slots(D, page, T):
    """Whatever the slots hold that no row sees, and whatever a call before left on the chip, a capped
    call's results are the same bit for bit (scores of both sides of the cap's polynomial range)."""
    B, H, Hkv, lens = 3, 8, 2, [100, 3, 333]
    wide = -(-max(lens) // page)
    g = torch.Generator().manual_seed(D)
    bt = torch.randperm(B * wide, generator=g).int().view(B, wide)
    q = rand((B, H, T, D), "bf16", 1, 2.0).cuda()
    pools = [rand((B * wide, Hkv, page, D), "bf16", s) for s in (2, 3)]
    free = torch.ones(B * wide, page, dtype=torch.bool)
    for b in range(B):
        for i in range(lens[b]):
            free[bt[b, i // page], i % page] = False
    noise = [rand((B * wide, Hkv, page, D), "bf16", s, 100.0).cuda() for s in (4, 5)]
    full = ints(*[wide * page] * B).cuda()
    first = None
    for fill in (0.0, 1e30, float("nan")):
        for x in pools:
            x.transpose(1, 2)[free] = fill
        kp, vp = (x.cuda() for x in pools)
        for window in (0, 77):
            for before in (1.0, 100.0):
                # leaves keys in shared memory that give large scores
                fa.paged_attention(q, noise[0] * before, noise[1], bt.cuda(), full)
                got = fa.paged_attention(q, kp, vp, bt.cuda(), ints(*lens).cuda(), softcap=20.0, window=window)
                first = first or {}
                want = first.setdefault(window, got)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (fill, window, before)


def test_append_reports_negative_counts():
    """A negative new_lens is outside 0 to T: nothing is written, and the status says so."""
    B, H, T, D, page = 2, 2, 2, 64, 16
    k = rand((B, H, T, D), "fp16", 1).cuda()
    for bad in (-1, -2 ** 31):
        kp, vp = (torch.zeros(2, H, page, D, dtype=torch.float16, device="cuda") for _ in range(2))
        out = fa.paged_append(k, k, kp, vp, ints(0, 1)[:, None].cuda(), ints(5, 5).cuda(), new_lens=ints(bad, 1).cuda(),
                              q=k, table=fa.rotary_table(16, 64).cuda())
        torch.cuda.synchronize()
        assert fa.fa_device_status(reset=True) == 13
        assert (kp[0] == 0).all() and (vp[0] == 0).all() and (out[0] == 0).all()
        assert torch.equal(vp[1, :, 4], k[1, :, 0]) and (out[1, :, 1] == 0).all()


@pytest.mark.parametrize("H,Hkv,N,D,cap,alibi,dtype", [
    (2, 2, 200, 64, 0.0, False, "bf16"), (4, 2, 300, 128, 30.0, False, "bf16"), (3, 1, 200, 96, 0.0, True, "bf16"),
    (2, 1, 260, 64, 20.0, True, "bf16"), (4, 1, 300, 128, 30.0, True, "fp16")])
def test_masked_rows_of_the_largest_values(H, Hkv, N, D, cap, alibi, dtype):
    """Padded rows that hold the type's largest and lowest values (their products with other rows leave
    the fp32 range): outputs and gradients of the other rows are those of padding with zeros."""
    q, k, v, do = (rand((2, h, N, D), dtype, s, 1.5) for s, h in enumerate((H, Hkv, Hkv, H)))
    ids = (torch.arange(N) * 3 // N).int().repeat(2, 1)
    ids[0, N - 70:] = -1
    ids[1, 40:90] = -1
    pad = ids < 0
    for t in (q, k, v, do):
        t.transpose(1, 2)[pad] = 0
    seen = ref.visible(2, N, documents=ids)
    slopes = torch.tensor([0.4 / (h + 1) for h in range(H)]) if alibi else None
    want, bound = ref.attention(q, k, v, do, 0.125, seen, cap, slopes)
    most = torch.finfo(DT[dtype]).max
    sign = torch.where(torch.arange(D) % 3 == 0, -most, most).to(DT[dtype])
    for fill in (torch.full((D,), -most, dtype=DT[dtype]), sign):
        for t in (q, k, v, do):
            t.transpose(1, 2)[pad] = fill
        qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
        more = dict(mask=fa.attention_mask(2, N, documents=ids.cuda()), softcap=cap,
                    alibi_slopes=None if slopes is None else slopes.cuda())
        o, lse = fa.attention_forward(qd, kd, vd, 0.125, **more)
        grads = fa.attention_backward(qd, kd, vd, o, lse, dod, 0.125, **more)
        for name, t in zip(("O", "lse", "dQ", "dK", "dV"), (o, lse, *grads)):
            ref.check(t, want[name], bound[name], name)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,cap", [(64, 0.0), (128, 0.0), (128, 20.0), (96, 3.0)])
def test_distance_bias_rows_of_one_key_return_its_value(D, cap, dtype):
    """A row that sees one key has P = 1: O is that key's value, bit for bit, whatever the slope."""
    B, H, N = 1, 4, 300
    q, k, v = (rand((B, H, N, D), dtype, s, 1.5).cuda() for s in range(3))
    slopes = torch.tensor([0.7, 0.31, 0.05, -0.4]).cuda()
    each = fa.attention_mask(B, N, documents=torch.arange(N, dtype=torch.int32)[None].cuda())
    o, _ = fa.attention_forward(q, k, v, mask=each, softcap=cap, alibi_slopes=slopes)
    assert torch.equal(o, v)
    o, _ = fa.attention_forward(q, k, v, causal=True, softcap=cap, alibi_slopes=slopes)
    assert torch.equal(o[:, :, 0], v[:, :, 0])


def test_distance_bias_keeps_small_weights():
    """fp16: keys that weigh 2^-18 of a row's largest count, next to slopes whose bias changes by 7 bits
    over eight columns (the largest weight is 2^-7 of the largest score with the least bias there)."""
    N, D, slope = 128, 64, 0.7
    i = N - 1
    q = torch.zeros(1, 1, N, D)
    q[..., 0] = 1.0
    k = torch.zeros(1, 1, N, D)
    away = (i - torch.arange(N)).double()
    k[0, 0, :, 0] = (slope * away - 18 * 0.6931).float()       # every key weighs 2^-18
    k[0, 0, i - 7, 0] = slope * 7                              # this one 1
    v = torch.full((1, 1, N, D), 100.0)
    v[0, 0, i - 7] = 1.0
    q, k, v = (t.half() for t in (q, k, v))
    slopes = torch.tensor([slope])
    want, bound = ref.attention(q, k, v, None, 1.0, ref.visible(1, N), 0.0, slopes)
    share = want["O"][0, 0, i, 0] - v[0, 0, i - 7, 0].double()
    assert share > 0.04 and bound["O"][0, 0, i, 0] < share / 8
    o, lse = fa.attention_forward(q.cuda(), k.cuda(), v.cuda(), 1.0, True, alibi_slopes=slopes.cuda())
    ref.check(o, want["O"], bound["O"])
    ref.check(lse, want["lse"], bound["lse"])


def test_windows_beyond_c_integers():
    """A window longer than any int limits nothing; one below every int is refused like any negative one."""
    N, D = 300, 64
    q, k, v = (rand((1, 2, N, D), "bf16", s).cuda() for s in range(3))
    want = fa.attention_forward(q, k, v, mask=fa.attention_mask(1, N, device="cuda"))
    here = torch.cuda.current_stream()
    kp, vp, bt = k[0].view(2, 1, 300, 64)[:, :, :256].contiguous(), v[0].view(2, 1, 300, 64)[:, :, :256].contiguous(), ints(0, 1)[None].cuda()
    sl, q1 = ints(400).cuda(), q[:, :, :1].contiguous()
    paged = fa.paged_attention(q1, kp, vp, bt, sl)
    for window in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63, 10 ** 30):
        for stream in (None, here):
            mask = fa.attention_mask(1, N, window=window, device="cuda", stream=stream)
            assert all(torch.equal(a, b) for a, b in zip(fa.attention_forward(q, k, v, mask=mask), want))
            got = fa.paged_attention(q1, kp, vp, bt, sl, window=window, stream=stream)
            assert all(torch.equal(a, b) for a, b in zip(got, paged))
    for window in (-1, -2 ** 32, -2 ** 32 + 5, -10 ** 30):
        with pytest.raises(fa.FAError):
            fa.attention_mask(1, N, window=window, device="cuda")
        with pytest.raises(fa.FAError):
            fa.paged_attention(q1, kp, vp, bt, sl, window=window)


def test_caps_outside_fp32_are_refused():
    """A cap that is 0 as a float would leave the scores uncapped, others would divide by nothing."""
    q = rand((1, 2, 40, 64), "bf16", 1).cuda()
    kp, bt, sl = q[0].view(2, 1, 40, 64)[:, :, :32].contiguous(), ints(0, 1)[None].cuda(), ints(50).cuda()
    here = torch.cuda.current_stream()
    for cap in (1e-50, 1e-45, 1e-40, 3e38, 1e39, -1e-50):
        for stream in (None, here):
            with pytest.raises(fa.FAError):
                fa.attention_forward(q, q, q, softcap=cap, stream=stream)
            with pytest.raises(fa.FAError):
                fa.attention_backward(q, q, q, q, q[..., 0].float(), q, softcap=cap, stream=stream)
            with pytest.raises(fa.FAError):
                fa.paged_attention(q[:, :, :1].contiguous(), kp, kp, bt, sl, softcap=cap, stream=stream)


@pytest.mark.parametrize("cap", [1e-36, 1e-20, 1e30, 2e38])
def test_caps_at_the_ends_of_fp32(cap):
    """The smallest caps leave equal weights, the largest the uncapped scores."""
    B, H, N, D = 1, 2, 150, 64
    q, k, v, do = (rand((B, H, N, D), "bf16", s) for s in range(4))
    want, bound = ref.attention(q, k, v, do, 0.125, ref.visible(B, N), cap if cap < 1 else 0.0)
    d = [t.cuda() for t in (q, k, v, do)]
    o, lse = fa.attention_forward(*d[:3], 0.125, True, softcap=cap)
    grads = fa.attention_backward(*d[:3], o, lse, d[3], 0.125, True, softcap=cap)
    for name, t in zip(("O", "lse", "dQ", "dK", "dV"), (o, lse, *grads)):
        ref.check(t, want[name], bound[name], name)
    page = 16
    kp, vp = (torch.nn.functional.pad(t, (0, 0, 0, 10)).view(B, H, 10, page, D).transpose(1, 2).flatten(0, 1).contiguous().cuda()
              for t in (k, v))
    o1, lse1 = fa.paged_attention(d[0][:, :, -1:].contiguous(), kp, vp, torch.arange(10, dtype=torch.int32)[None].cuda(),
                                  ints(N).cuda(), 0.125, softcap=cap)
    ref.check(o1, want["O"][:, :, -1:], bound["O"][:, :, -1:])
    ref.check(lse1, want["lse"][:, :, -1:], bound["lse"][:, :, -1:])


def test_out_of_memory_is_torchs_own_error():
    """Outputs larger than the card, through both host paths: torch.OutOfMemoryError, and the next call works."""
    x = rand((1, 1, 1, 256), "bf16", 1).cuda()
    huge = x.expand(64, 64, 1 << 18, 256)                       # 550 GB as a contiguous result
    table = fa.rotary_table(8, 256).cuda()
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(torch.OutOfMemoryError):
            fa.rotary_forward(huge, None, table, stream=stream)
    assert torch.equal(fa.rotary_forward(x, None, table)[0], x)  # position 0 turns by nothing


def test_results_without_the_module_of_the_small_calls(monkeypatch):
    """Every operator through the Python path alone: the same results."""
    B, H, Hkv, N, D = 2, 4, 2, 60, 64
    q, k, v, do = (rand((B, h, N, D), "fp16", s).cuda() for s, h in enumerate((H, Hkv, Hkv, H)))
    table, ids = fa.rotary_table(N, D).cuda(), (torch.arange(N) // 25).int().repeat(B, 1).cuda()
    bt = torch.arange(8, dtype=torch.int32).view(B, 4).cuda()

    def step():
        mask = fa.attention_mask(B, N, documents=ids)
        out = fa.attention_forward(q, k, v, mask=mask, softcap=10.0)
        dq, dk, dv = fa.attention_backward(q, k, v, *out, do, mask=mask, softcap=10.0)
        kp, vp = (torch.zeros(8, Hkv, 16, D, dtype=torch.float16, device="cuda") for _ in range(2))
        qn = fa.paged_append(k, v, kp, vp, bt, ints(N, N).cuda(), q=q, table=table)
        last = fa.paged_attention(qn[:, :, -1:].contiguous(), kp, vp, bt, ints(N, N).cuda())
        return (*out, dk, dv, qn, kp, vp, *last, *fa.rotary_forward(q, k, table))

    fa.load_library()
    assert base._fast is not None
    want = step()
    monkeypatch.setattr(base, "_fast", None)
    assert all(torch.equal(a, b) for a, b in zip(step(), want))


@pytest.mark.parametrize("how", ["argument", "context"])
def test_a_mask_may_be_dropped_while_another_stream_reads_it(how):
    """The plan's memory is not handed out again before the call on the other stream has run."""
    B, N = 1, 4096
    q, k, v, do = (rand((B, 1, N, 64), "bf16", s).cuda() for s in range(4))
    o, lse = fa.attention_forward(q, k, v, mask=fa.attention_mask(B, N, device="cuda", window=100))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda m, s: fa.attention_forward(q, k, v, mask=m, stream=s),
                 lambda m, s: fa.attention_backward(q, k, v, o, lse, do, mask=m, stream=s)):
        torch.cuda.empty_cache()
        mask = fa.attention_mask(B, N, device="cuda", window=100)
        at, size = mask.plan.data_ptr(), mask.plan.numel()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000_000)                    # half a second
            if how == "context":
                out = call(mask, None)
        if how == "argument":
            out = call(mask, side)
        del mask
        others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
        busy = not side.query()
        assert busy and at not in [t.data_ptr() for t in others]
        torch.cuda.synchronize()
        del out, others


def outcome(call):
    try:
        r = call()
    except Exception as e:                                      # noqa: BLE001 - its type and text are compared
        return type(e), str(e)
    return [None if t is None else torch.nan_to_num(t.float()).cpu() for t in (r if isinstance(r, tuple) else (r,))]


def test_both_host_paths_accept_and_refuse_alike(monkeypatch):
    """Calls near the edge of what is allowed: the C++ marshalling and the Python path take the same
    ones, with the same results, and refuse the others with the same error."""
    B, H, Hkv, N, D, page = 2, 4, 2, 20, 64, 16
    q, k, v, do = (rand((B, h, N, D), "bf16", s).cuda() for s, h in enumerate((H, Hkv, Hkv, H)))
    table, pos = fa.rotary_table(N, D).cuda(), torch.arange(N, dtype=torch.int32, device="cuda")
    slopes = torch.ones(H, device="cuda")
    kp, vp = (rand((6, Hkv, page, D), "bf16", s).cuda() for s in (5, 6))
    bt, sl = torch.arange(6, dtype=torch.int32).view(B, 3).cuda(), ints(20, 33).cuda()
    o, lse = fa.attention_forward(q, k, v, causal=True)
    ids = torch.zeros(B, N, dtype=torch.int32, device="cuda")
    mask = fa.attention_mask(B, N, documents=ids)
    wide = torch.zeros(B, H, N, 80, dtype=torch.bfloat16, device="cuda")
    param = torch.nn.Parameter(q.clone())
    cpu = q.cpu()
    rotary = [dict(), dict(positions=pos), dict(positions=pos[None]), dict(positions=pos.expand(B, N)),
              dict(positions=pos.repeat(B, 1)), dict(positions=pos[:-1]), dict(positions=pos.long()), dict(positions=pos.cpu()),
              dict(positions=pos[None, None]), dict(positions=pos.repeat(3, 1)), dict(positions=0), dict(interleaved=1),
              dict(interleaved=2), dict(interleaved=None), dict(table=table[:, :32].contiguous()), dict(table=table[:, ::2]),
              dict(table=table[:0]), dict(table=table[0]), dict(table=table.double()), dict(table=None), dict(table=table.cpu()),
              dict(q=None), dict(k=None), dict(q=None, k=None), dict(q=param), dict(q=cpu), dict(q=q[0]), dict(q=q.float()),
              dict(q=q.half()), dict(k=k[:1]), dict(k=k[:, :0]), dict(q=q[:, :, :0], k=k[:, :, :0]), dict(k=k[..., :32]),
              dict(q=wide[..., 8:72]), dict(q=wide[..., 4:68]), dict(q=wide[..., :64].transpose(1, 2)), dict(q=q[:, :1].expand(B, H, N, D)),
              dict(q=q.flip(2)), dict(q=wide, k=None), dict(q=1)]
    att = [dict(), dict(causal=True), dict(causal=1), dict(causal=2), dict(causal=None), dict(mask=mask), dict(mask=mask, causal=True),
           dict(mask=mask.plan), dict(mask=fa.attention_mask(1, N, documents=ids[:1])), dict(softcap=5), dict(softcap=5.0), dict(softcap=True),
           dict(softcap=-5.0), dict(softcap="5"), dict(scale=1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=10 ** 400),
           dict(alibi_slopes=slopes), dict(alibi_slopes=slopes[:2]), dict(alibi_slopes=slopes.half()), dict(alibi_slopes=slopes[None]),
           dict(alibi_slopes=slopes.cpu()), dict(q=param), dict(k=k.half()), dict(k=cpu), dict(v=v[:, :1]), dict(v=v[..., :32]),
           dict(q=q[:, :3].contiguous()), dict(q=q.transpose(1, 2)), dict(k=k[:, :0], v=v[:, :0]), dict(q=q.float(), k=k.float(), v=v.float()),
           dict(q=wide, k=wide[:, :2].contiguous(), v=wide[:, :2].contiguous())]
    back = [dict(), dict(o=o[:1]), dict(lse=lse[:, :1]), dict(lse=lse.half()), dict(do=do.half()), dict(do=do.transpose(1, 2)),
            dict(do=do[..., :32]), dict(o=o.cpu())]
    new = k[:, :, :3].contiguous()
    append = [dict(), dict(new_lens=ints(1, 3).cuda()), dict(new_lens=ints(1, 3)), dict(new_lens=ints(1).cuda()), dict(new_lens=2),
              dict(q=q[:, :, :3].contiguous()), dict(q=q[:, :, :3]), dict(q=q), dict(q=q[:, :, :3], table=None), dict(table=None),
              dict(table=table[:, :40]), dict(k=new[:1]), dict(k=k[:, :, :3]), dict(v=new.half()), dict(k_pages=kp[:, :1].contiguous()),
              dict(k_pages=kp[:, :, :12].contiguous(), v_pages=vp[:, :, :12].contiguous()), dict(k_pages=kp.transpose(1, 2)),
              dict(v_pages=vp.cpu()), dict(k_pages=kp[:0], v_pages=vp[:0]), dict(block_table=bt[:1]), dict(block_table=bt[:, :0]), dict(block_table=bt.long()),
              dict(seq_lens=sl[:1]), dict(seq_lens=sl[None]), dict(seq_lens=sl.long()), dict(interleaved=True), dict(interleaved=3),
              dict(k=new[:, :, :0], v=new[:, :, :0]), dict(k=torch.nn.Parameter(new))]
    q1 = q[:, :, :2].contiguous()
    decode = [dict(), dict(softcap=3), dict(softcap=None), dict(scale=None), dict(scale=-1.0), dict(window=3), dict(window=True), dict(window=-1), dict(window=2.0),
              dict(window=None), dict(alibi_slopes=slopes), dict(alibi_slopes=slopes[:1]), dict(alibi_slopes=slopes.double()), dict(q=q[:, :, :2]),
              dict(q=q1[:1]), dict(q=q1[0]), dict(q=q1.float()), dict(q=q1.half()), dict(q=q1[:, :3].contiguous()), dict(q=q1[:, :, :0]), dict(q=torch.nn.Parameter(q1)),
              dict(k_pages=kp[..., :32]), dict(v_pages=vp[:, :1].contiguous()), dict(k_pages=kp[:, :, :12].contiguous(), v_pages=vp[:, :, :12].contiguous()),
              dict(block_table=bt[0]), dict(block_table=bt[:, :2]), dict(block_table=bt[:, :0].contiguous()), dict(seq_lens=sl[:1]), dict(seq_lens=sl.cpu())]
    masks = [dict(), dict(documents=ids), dict(documents=ids[:1]), dict(documents=ids.long()), dict(documents=ids.t()), dict(documents=ids.cpu()),
             dict(prefix=ints(3, 4).cuda()), dict(prefix=ints(3).cuda()), dict(prefix=ints(3, 4).cuda(), causal=False), dict(prefix=ints(3, 4).cuda(), window=2),
             dict(prefix=ints(3, 4).cuda(), documents=ids), dict(window=3), dict(window=-3), dict(window=2.0), dict(window=True), dict(window=None), dict(causal=0),
             dict(causal=5), dict(causal=False, window=2), dict(B=0), dict(N=0), dict(N=1 << 19), dict(B=2.0), dict(device="cuda:0"), dict(device="cpu")]

    def rows(plan):
        n = 2 * B * 128                                          # behind the intervals: unused entries
        return plan.view(torch.int32)[:n].clone()

    def turned(q=q, k=k, table=table, **kw):
        return fa.rotary_forward(q, k, table, **kw)

    def attended(q=q, k=k, v=v, scale=None, causal=False, **kw):
        return fa.attention_forward(q, k, v, scale, causal, **kw)

    def gradients(o=o, lse=lse, do=do):
        return fa.attention_backward(q, k, v, o, lse, do, causal=True)[1:]

    def appended(k=new, v=new, k_pages=kp, v_pages=vp, block_table=bt, seq_lens=sl, table=table, **kw):
        out = fa.paged_append(k, v, k_pages, v_pages, block_table, seq_lens, table=table, **kw)
        return out, k_pages, v_pages

    def decoded(q=q1, k_pages=kp, v_pages=vp, block_table=bt, seq_lens=sl, **kw):
        return fa.paged_attention(q, k_pages, v_pages, block_table, seq_lens, **kw)

    def planned(B=B, N=N, **kw):
        return rows(fa.attention_mask(B, N, **{"device": "cuda", **kw}).plan)

    took = 0
    for f, cases in ((turned, rotary), (attended, att), (gradients, back), (appended, append), (decoded, decode), (planned, masks)):
        for kw in cases:
            with monkeypatch.context() as m:
                pools = kp.clone(), vp.clone()
                a = outcome(lambda: f(**kw))
                kp.copy_(pools[0]), vp.copy_(pools[1])
                m.setattr(base, "_fast", None)
                b = outcome(lambda: f(**kw))
                kp.copy_(pools[0]), vp.copy_(pools[1])
            fa.fa_device_status(reset=True)
            what = f.__name__, {n: tuple(x.shape) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
            if isinstance(a, tuple) or isinstance(b, tuple):
                assert a == b, (what, a, b)
            else:
                took += 1
                assert len(a) == len(b) and all((x is y) or torch.equal(x, y) for x, y in zip(a, b)), what
    assert took >= 40


@pytest.mark.parametrize("H,Hkv,T,lens,page,cap,window,dtype", [
    (16, 1, 5, [700, 80], 32, 0.0, 0, "bf16"),                  # 80 rows: three groups
    (9, 1, 11, [1500, 7, 128], 16, 20.0, 300, "fp16"),           # 99: four, the last of three rows
    (24, 2, 64, [64, 500], 128, 0.0, 0, "bf16"),                 # 768: the most tokens
])
def test_decode_several_groups_of_rows_at_256_columns(H, Hkv, T, lens, page, cap, window, dtype):
    B, D, wide = len(lens), 256, -(-max(lens) // page)
    q = rand((B, H, T, D), dtype, 1, 2.0)
    kp, vp = (rand((B * wide, Hkv, page, D), dtype, s) for s in (2, 3))
    bt = torch.randperm(B * wide, generator=torch.Generator().manual_seed(4)).int().view(B, wide)
    want = ref.paged_attention(q, kp, vp, bt, ints(*lens), ref.default_scale(D), cap, None, window)
    o, l = fa.paged_attention(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), ints(*lens).cuda(), softcap=cap, window=window)
    ref.check(o, want[0], want[2], "O")
    ref.check(l, want[1], want[3], "lse")


@pytest.mark.parametrize("B,H,Hkv,N,D,kind,cap,alibi,dtype", [
    (1, 3, 1, 450, 128, "causal", 0.0, False, "bf16"), (1, 5, 1, 400, 96, "documents", 0.0, False, "bf16"),
    (2, 3, 1, 500, 128, "documents", 30.0, False, "fp16"), (1, 6, 2, 450, 128, "full", 0.0, True, "bf16"),
    (1, 5, 1, 420, 64, "documents", 0.0, True, "fp16"), (1, 9, 3, 390, 96, "causal", 20.0, True, "bf16")])
def test_odd_groups_walk_all_their_heads(B, H, Hkv, N, D, kind, cap, alibi, dtype):
    """Groups of 3 and 5 query heads with several query tiles each: one CTA goes from head to head."""
    q, k, v, do = (rand((B, h, N, D), dtype, s, 1.5) for s, h in enumerate((H, Hkv, Hkv, H)))
    ids = (torch.arange(N) * 4 // N).int().repeat(B, 1)
    ids[:, N - 30:] = -1
    slopes = torch.tensor([0.5 / (h + 1) for h in range(H)]) if alibi else None
    seen = ref.visible(B, N, documents=ids) if kind == "documents" else ref.visible(B, N, causal=kind == "causal")
    want, bound = ref.attention(q, k, v, do, 0.09, seen, cap, slopes)
    d = [t.cuda() for t in (q, k, v, do)]
    more = dict(mask=fa.attention_mask(B, N, documents=ids.cuda()) if kind == "documents" else None, softcap=cap,
                alibi_slopes=None if slopes is None else slopes.cuda())
    o, lse = fa.attention_forward(*d[:3], 0.09, kind == "causal", **more)
    grads = fa.attention_backward(*d[:3], o, lse, d[3], 0.09, kind == "causal", **more)
    for name, t in zip(("O", "lse", "dQ", "dK", "dV"), (o, lse, *grads)):
        ref.check(t, want[name], bound[name], name)


@pytest.mark.parametrize("D,causal,cap", [(128, True, 0.0), (96, False, 20.0)])
def test_many_items_walk_even_groups_in_one_cta(D, causal, cap):
    """Enough key tiles that pairs of heads are not split over CTAs (four items an SM): two of the
    key-value heads against the 64-bit form."""
    B, H, Hkv, N = 5, 64, 32, 400
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v, do = (torch.randn(B, h, N, D, generator=g, device="cuda").bfloat16() for h in (H, Hkv, Hkv, H))
    o, lse = fa.attention_forward(q, k, v, causal=causal, softcap=cap)
    dq, dk, dv = fa.attention_backward(q, k, v, o, lse, do, causal=causal, softcap=cap)
    for b, h in ((0, 0), (4, 31)):
        two, one = (slice(b, b + 1), slice(2 * h, 2 * h + 2)), (slice(b, b + 1), slice(h, h + 1))
        want, bound = ref.attention(*(t[i].cpu() for t, i in ((q, two), (k, one), (v, one), (do, two))), ref.default_scale(D),
                                    ref.visible(1, N, causal=causal), cap)
        for name, t, i in (("O", o, two), ("lse", lse, two), ("dQ", dq, two), ("dK", dk, one), ("dV", dv, one)):
            ref.check(t[i], want[name], bound[name], name)
