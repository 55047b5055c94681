"""Score-modified attention on the GPU (mask plan, forward, backward, autograd) against the 64-bit
form, element by element."""
import threading

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


def documents(B, N, kind):
    g = torch.Generator().manual_seed(N)
    ids = torch.zeros(B, N, dtype=torch.int32)
    for b in range(B):
        if kind == "each":                       # every row its own document
            ids[b] = torch.arange(N)
        elif kind == "padded":                   # runs, a padded middle and tail; the last batch row all padding
            cuts = torch.randint(0, 2, (N,), generator=g).mul_(torch.randint(0, 3, (N,), generator=g) == 0).cumsum(0)
            ids[b] = cuts.int()
            ids[b, N // 3: N // 3 + max(1, N // 9)] = -1
            ids[b, N - N // 4:] = -5
            if b == B - 1 and B > 1:
                ids[b] = -1
        else:                                    # a few long runs; an id that comes back is another run
            ids[b] = (torch.arange(N) * 5 // N) % 3
    return ids


def mask_args(kind, B, N):
    """(arguments of attention_mask or None, causal argument of the call, dense visibility)"""
    if kind in ("full", "causal", "hot", "steep", "steep-full"):
        causal = kind in ("causal", "hot", "steep")
        return None, causal, ref.visible(B, N, causal=causal)
    if kind.startswith("doc"):
        _, which, *rest = kind.split("-")
        a = dict(documents=documents(B, N, which), causal="full" not in rest)
    elif kind.startswith("prefix"):
        a = dict(prefix=torch.tensor([[0, N, N // 2, -3, N + 9, 1][(b + len(kind)) % 6] for b in range(B)], dtype=torch.int32))
    else:
        w, *rest = kind[6:].split("-")
        a = dict(window=N + 7 if w == "N" else int(w), causal="full" not in rest)
    return a, False, ref.visible(B, N, **a)


CASES = [
    # B, H, Hkv, N, D, mask, softcap, alibi, dtype
    (1, 1, 1, 1, 64, "causal", 0.0, False, "bf16"),
    (2, 4, 2, 1, 128, "full", 30.0, True, "fp16"),
    (1, 2, 1, 2, 32, "full", 0.0, False, "fp16"),
    (2, 3, 1, 5, 96, "doc-each", 20.0, False, "bf16"),
    (1, 4, 2, 127, 64, "causal", 0.0, False, "bf16"),
    (1, 4, 1, 128, 128, "full", 0.0, True, "bf16"),
    (2, 5, 1, 129, 64, "doc-padded", 0.0, False, "fp16"),
    (3, 2, 2, 300, 128, "doc-padded", 30.0, False, "bf16"),
    (2, 4, 2, 384, 96, "doc-padded-full", 0.0, True, "fp16"),
    (2, 6, 2, 513, 64, "doc-long", 50.0, True, "bf16"),
    (2, 4, 4, 640, 128, "doc-long-full", 0.0, False, "bf16"),
    (1, 2, 1, 260, 64, "doc-each", 0.0, False, "bf16"),
    (6, 2, 1, 257, 64, "prefix", 0.0, False, "bf16"),
    (6, 2, 2, 400, 128, "prefixed", 15.0, True, "fp16"),
    (1, 2, 1, 300, 128, "window1", 0.0, False, "bf16"),
    (1, 4, 2, 700, 64, "window130", 0.0, True, "fp16"),
    (2, 2, 2, 515, 128, "window64-full", 30.0, False, "bf16"),
    (1, 3, 3, 200, 96, "windowN", 0.0, False, "bf16"),
    (1, 2, 1, 200, 32, "windowN-full", 5.0, False, "fp16"),
    (1, 8, 1, 256, 128, "causal", 30.0, False, "bf16"),
    (1, 8, 2, 385, 64, "full", 0.0, False, "fp16"),
    # more work items than SMs: one CTA for all heads of a group
    (5, 20, 10, 300, 64, "doc-padded", 0.0, False, "bf16"),
    # scores far beyond the cap (the other way to its tanh), and steep slopes
    (1, 4, 2, 300, 128, "hot", 5.0, False, "bf16"),
    (1, 4, 2, 300, 64, "hot", 3.0, True, "fp16"),
    (1, 2, 2, 400, 64, "steep", 0.0, True, "fp16"),
    (1, 2, 1, 300, 128, "steep-full", 20.0, True, "bf16"),
    # caps whose polynomial leaves the floats' range, and tiny ones
    (1, 2, 1, 200, 64, "causal", 2e4, False, "fp16"),
    (1, 2, 2, 200, 128, "full", 1e9, True, "bf16"),
    (1, 2, 2, 200, 64, "full", 1e-3, False, "bf16"),
    (1, 2, 1, 260, 128, "window100-full", 0.2, True, "fp16"),
]


def inputs(B, H, Hkv, N, D, dtype, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda h, s=1.0: (torch.randn(B, h, N, D, generator=g) * s).to(DT[dtype])
    return r(H, std), r(Hkv), r(Hkv), r(H)


def slopes_of(H, alibi):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]) if alibi else None


@pytest.mark.parametrize("B,H,Hkv,N,D,kind,cap,alibi,dtype", CASES)
def test_forward_and_gradients(B, H, Hkv, N, D, kind, cap, alibi, dtype):
    q, k, v, do = inputs(B, H, Hkv, N, D, dtype, N + D, 8.0 if kind == "hot" else 1.5)
    args, causal, seen = mask_args(kind, B, N)
    slopes, scale = slopes_of(H, alibi), ref.default_scale(D)
    if kind.startswith("steep"):
        slopes = torch.tensor([3.0, -0.02])
    want, bound = ref.attention(q, k, v, do, scale, seen, cap, slopes)
    cu = lambda t: None if t is None else t.cuda()
    qd, kd, vd, dod, sd = cu(q), cu(k), cu(v), cu(do), cu(slopes)
    mask = None
    if args is not None:
        mask = fa.attention_mask(B, N, **{n: cu(x) if isinstance(x, torch.Tensor) else x for n, x in args.items()})
    more = dict(mask=mask, softcap=cap, alibi_slopes=sd)
    if mask is None and not cap and sd is None and H == Hkv:
        o, lse = torch.empty_like(qd), torch.empty(B, H, N, device="cuda")
        fa.fa_fwd_mod(qd, kd, vd, o, lse, scale, causal)
        grads = [torch.empty_like(t) for t in (qd, kd, vd)]
        ws = torch.empty(fa.fa_bwd_workspace_size(B, H, N, D), device="cuda", dtype=torch.uint8)
        fa.fa_bwd_mod(qd, kd, vd, o, dod, lse, *grads, ws, scale, causal)
    else:
        o, lse = fa.attention_forward(qd, kd, vd, scale, causal, **more)
        grads = fa.attention_backward(qd, kd, vd, o, lse, dod, scale, causal, **more)
    torch.cuda.synchronize()
    for name, t in zip(("O", "lse", "dQ", "dK", "dV"), (o, lse, *grads)):
        ref.check(t, want[name], bound[name], (name, kind))


@pytest.mark.parametrize("kind", ["doc-padded", "doc-long-full", "doc-each", "prefix", "window3", "window200-full", "windowN"])
@pytest.mark.parametrize("B,N", [(1, 1), (2, 33), (6, 128), (2, 1000), (1, 5000)])
def test_mask_plan_rows(kind, B, N):
    """The plan's intervals are the definition's, and its tile ranges hold every visible pair."""
    args, _, seen = mask_args(kind, B, N)
    mask = fa.attention_mask(B, N, device="cuda",
                             **{n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in args.items()})
    plan = mask.plan.view(torch.int32).cpu()
    npad = -(-N // 128) * 128
    rows = plan[: 2 * B * npad].view(B, npad, 2)
    j = torch.arange(N)
    dense = (j >= rows[:, :N, :1]) & (j < rows[:, :N, 1:])
    assert torch.equal(dense, seen)
    assert (rows[:, N:] == 0).all()
    nt = npad // 128
    tiles = plan[2 * B * npad: 2 * B * npad + 4 * B * nt].view(B, nt, 4)
    order = plan[2 * B * npad + 4 * B * nt:].view(B, nt, 2)
    pad = torch.zeros(B, npad, npad, dtype=torch.bool)
    pad[:, :N, :N] = seen
    blocks = pad.view(B, nt, 128, nt, 128).any(4).any(2)
    t = torch.arange(nt)
    by_query = (t >= tiles[:, :, :1]) & (t < tiles[:, :, 1:2])
    by_key = (t >= tiles[:, :, 2:3]) & (t < tiles[:, :, 3:])
    assert not (blocks & ~by_query).any() and not (blocks.transpose(1, 2) & ~by_key).any()
    # every key tile and query block once, those with most work first
    work_k, work_q = tiles[..., 3] - tiles[..., 2], tiles[..., 1] - tiles[..., 0]
    work_q = torch.nn.functional.pad(work_q, (0, nt % 2)).view(B, -1, 2).sum(-1)
    for items, work in ((order[..., 0], work_k), (order[:, : work_q.shape[1], 1], work_q)):
        assert torch.equal(items.sort(-1).values, torch.arange(items.shape[1], dtype=torch.int32).expand_as(items))
        assert (work.gather(1, items.long()).diff(dim=1) <= 0).all()


def test_unmodified_call_keeps_its_path():
    q, k, v, _ = (t.cuda() for t in inputs(1, 2, 2, 300, 64, "bf16", 3))
    o, lse = fa.attention_forward(q, k, v, 0.125, True)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    fa.fa_fwd(q, k, v, o2, lse2, 0.125, True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_long_window_is_no_window():
    """A window longer than the sequence gives the causal plan's results bit for bit."""
    q, k, v, do = (t.cuda() for t in inputs(2, 2, 2, 500, 128, "bf16", 4))
    masks = [fa.attention_mask(2, 500, window=w, device="cuda") for w in (0, 500, 1000, 2 ** 31 - 1)]
    outs = [fa.attention_forward(q, k, v, 0.09, mask=m) for m in masks]
    assert all(torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1]) for o, l in outs[1:])


def test_masked_rows_leave_neighbours_alone():
    """Large finite values (the type's largest) in padded rows change nothing elsewhere."""
    B, H, N, D = 1, 2, 200, 64
    q, k, v, do = inputs(B, H, H, N, D, "bf16", 5)
    ids = torch.zeros(B, N, dtype=torch.int32)
    ids[:, 150:] = -1
    mask = fa.attention_mask(B, N, documents=ids.cuda())
    outs = []
    for big in (0.0, 1e30):
        t = [x.clone() for x in (q, k, v, do)]
        for x in t[:3]:
            x[:, :, 150:] = big
        t[3][:, :, 150:] = 1.0 if big else 0.0
        qd, kd, vd, dod = (x.cuda() for x in t)
        o, lse = fa.attention_forward(qd, kd, vd, 0.125, mask=mask)
        g = fa.attention_backward(qd, kd, vd, o, lse, dod, 0.125, mask=mask)
        assert (o[:, :, 150:] == 0).all() and (lse[:, :, 150:] == float("-inf")).all()
        assert all((x[:, :, 150:] == 0).all() for x in g)
        outs.append((o, lse) + g[1:])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_autograd_matches_the_calls():
    B, H, Hkv, N, D = 2, 4, 2, 200, 64
    q, k, v, do = (t.cuda() for t in inputs(B, H, Hkv, N, D, "bf16", 6))
    mask = fa.attention_mask(B, N, documents=documents(B, N, "padded").cuda())
    slopes = slopes_of(H, True).cuda()
    more = dict(mask=mask, softcap=20.0, alibi_slopes=slopes)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    out = fa.flash_attention(*leaves, **more)
    out.backward(do)
    o, lse = fa.attention_forward(q, k, v, **more)
    dq, dk, dv = fa.attention_backward(q, k, v, o, lse, do, **more)
    assert torch.equal(out, o) and torch.equal(leaves[1].grad, dk) and torch.equal(leaves[2].grad, dv)
    # dQ is summed in varying order: within two fp32 sums' difference, one step of the 16-bit result
    assert ((leaves[0].grad - dq).abs() <= 2 ** -7 * dq.abs() + 1e-6).all()
    with pytest.raises(ValueError):
        fa.flash_attention(*leaves, alibi_slopes=slopes.clone().requires_grad_())


def test_first_call_of_a_fresh_thread():
    """A thread whose first CUDA work is one of the library's calls (as an autograd thread's may be)."""
    B, H, N, D = 1, 2, 200, 64
    q, k, v, do = (t.cuda() for t in inputs(B, H, H, N, D, "bf16", 8))
    o, lse, dq, dk, dv, o2, lse2 = (torch.empty_like(t) for t in (q, q[..., 0].float(), q, k, v, q, q[..., 0].float()))
    ws = torch.empty(fa.fa_bwd_workspace_size(B, H, N, D), device="cuda", dtype=torch.uint8)
    stream = torch.cuda.current_stream().cuda_stream
    failed = []

    def run(call):
        try:
            call()
        except Exception as e:                      # noqa: BLE001 - handed to the test's thread
            failed.append(e)

    code = lambda name, *args: base._raise(getattr(fa.load_library(), name)(*args), name)
    p = base._p
    for call in (lambda: code("fa_fwd_mod", p(q), p(k), p(v), p(o), p(lse), None, None, 30.0, B, H, H, N, D, 0.125, 1, 0, stream),
                 lambda: code("fa_bwd_mod", p(q), p(k), p(v), p(o), p(do), p(lse), p(dq), p(dk), p(dv), p(ws),
                              ws.numel(), None, None, 30.0, B, H, H, N, D, 0.125, 1, 0, stream),
                 lambda: code("fa_fwd", p(q), p(k), p(v), p(o2), p(lse2), B, H, N, D, 0.125, 1, stream)):
        t = threading.Thread(target=run, args=(call,))
        t.start()
        t.join()
    assert not failed, failed
    want = fa.attention_forward(q, k, v, 0.125, True, softcap=30.0)
    grads = fa.attention_backward(q, k, v, *want, do, 0.125, True, softcap=30.0)
    assert torch.equal(o, want[0]) and torch.equal(dk, grads[1]) and torch.equal(dv, grads[2])
    assert torch.equal(o2, fa.attention_forward(q, k, v, 0.125, True)[0])


def test_streams_and_graph():
    """On another stream, and captured: the mask plan, forward and backward of one step."""
    B, H, Hkv, N, D = 1, 4, 1, 320, 128
    q, k, v, do = (t.cuda() for t in inputs(B, H, Hkv, N, D, "fp16", 7))
    ids = documents(B, N, "long").cuda()

    def step(stream=None):
        mask = fa.attention_mask(B, N, documents=ids, stream=stream)
        o, lse = fa.attention_forward(q, k, v, mask=mask, softcap=30.0, stream=stream)
        return (o, lse) + fa.attention_backward(q, k, v, o, lse, do, mask=mask, softcap=30.0, stream=stream)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = step(stream)
        torch.cuda.current_stream().wait_stream(side)
        for i in (0, 1, 3, 4):
            assert torch.equal(got[i], want[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    ids.copy_(documents(B, N, "padded"))
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    fresh = step()
    for i in (0, 1, 3, 4):
        assert torch.equal(got[i], fresh[i])
    assert ((got[2] - fresh[2]).abs() <= 2 ** -10 * fresh[2].abs() + 1e-6).all()


@pytest.mark.parametrize("kind,cap,alibi,dtype", [("doc-padded", 0.0, False, "bf16"), ("causal", 30.0, True, "fp16"),
                                                  ("prefix", 0.0, True, "bf16"), ("full", 2.0, False, "bf16")])
def test_both_host_paths_agree(kind, cap, alibi, dtype):
    """The call marshalled in C++ and the one marshalled in Python (a workspace given, another stream)."""
    B, H, Hkv, N, D = 2, 4, 2, 190, 64
    q, k, v, do = (t.cuda() for t in inputs(B, H, Hkv, N, D, dtype, 9))
    args, causal, _ = mask_args(kind, B, N)
    more = dict(softcap=cap, alibi_slopes=None if not alibi else slopes_of(H, True).cuda())
    if args is not None:
        more["mask"] = fa.attention_mask(B, N, device="cuda", **{n: x.cuda() if isinstance(x, torch.Tensor) else x
                                                               for n, x in args.items()})
    here = torch.cuda.current_stream()
    if args is not None:
        other = fa.attention_mask(B, N, device="cuda", stream=here, **{n: x.cuda() if isinstance(x, torch.Tensor) else x
                                                                      for n, x in args.items()})
        used = 8 * (128 + 2) * B * (-(-N // 128))       # past the orders' unused entries nothing is written
        assert torch.equal(more["mask"].plan[:used], other.plan[:used])
    a, b = fa.attention_forward(q, k, v, 0.2, causal, **more), fa.attention_forward(q, k, v, 0.2, causal, here, **more)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ws = torch.empty(fa.fa_bwd_workspace_size(B, H, N, D), device="cuda", dtype=torch.uint8)
    ga = fa.attention_backward(q, k, v, *a, do, 0.2, causal, **more)
    gb = fa.attention_backward(q, k, v, *a, do, 0.2, causal, workspace=ws, **more)
    assert torch.equal(ga[1], gb[1]) and torch.equal(ga[2], gb[2])


def test_refusals_with_gpu_tensors():
    """What the C++ path hands back is refused by the Python path, with its messages."""
    q, k, v, do = (t.cuda() for t in inputs(1, 4, 2, 64, 64, "bf16", 1))
    o, lse = fa.attention_forward(q, k, v, causal=True)
    mask = fa.attention_mask(1, 64, device="cuda")
    slopes = torch.ones(4, device="cuda")
    for error, call in [
        (TypeError, lambda: fa.attention_forward(q.float(), k.float(), v.float())),
        (TypeError, lambda: fa.attention_forward(q, k.half(), v)),
        (ValueError, lambda: fa.attention_forward(q, k, v[:, :1])),
        (ValueError, lambda: fa.attention_forward(q.transpose(1, 2).contiguous().transpose(1, 2), k, v)),
        (ValueError, lambda: fa.attention_forward(q, k, v, alibi_slopes=slopes[:2])),
        (TypeError, lambda: fa.attention_forward(q, k, v, alibi_slopes=slopes.double())),
        (ValueError, lambda: fa.attention_forward(q, k, v, mask=fa.attention_mask(1, 65, device="cuda"))),
        (ValueError, lambda: fa.attention_forward(q, k, v, causal=True, mask=mask)),
        (TypeError, lambda: fa.attention_forward(q, k, v, mask=mask.plan)),
        (fa.FAError, lambda: fa.attention_forward(q, k, v, softcap=-1.0)),
        (fa.FAError, lambda: fa.attention_forward(q[:, :3].contiguous(), k, v)),
        (fa.FAError, lambda: fa.attention_forward(q, k, v, -0.1)),
        (ValueError, lambda: fa.attention_backward(q, k, v, o, lse[:, :2], do)),
        (ValueError, lambda: fa.attention_backward(q, k, v, o, lse, do.transpose(1, 2))),
        (ValueError, lambda: fa.attention_backward(q, k, v, o, lse, do, deterministic=True)),
    ]:
        with pytest.raises(error):
            call()
    ids = torch.zeros(2, 16, dtype=torch.int32, device="cuda")
    for error, kw in [
        (ValueError, dict(documents=ids[:1])), (TypeError, dict(documents=ids.long())), (ValueError, dict(documents=ids.cpu())),
        (fa.FAError, dict(prefix=ids[:, 0].contiguous(), causal=False)), (fa.FAError, dict(window=-1, device="cuda")),
        (fa.FAError, dict(prefix=ids[:, 0].contiguous(), window=3)), (ValueError, dict(prefix=ids[0])),
    ]:
        with pytest.raises(error):
            fa.attention_mask(2, 16, **kw)
    for B, N in ((0, 4), (1, 0), (1, 262145)):
        with pytest.raises(fa.FAError):
            fa.attention_mask(B, N, device="cuda")
    wide = torch.zeros(1, 2, 16, 256, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(fa.FAError):
        fa.attention_forward(wide, wide, wide, softcap=1.0)


@pytest.mark.parametrize("N,args", [(262144, dict(window=900)), (200001, "documents")])
def test_longest_sequences(N, args):
    """The longest plan: sampled rows of the forward and of dQ against 64 bits."""
    H, D, cap = 2, 64, 20.0
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn(1, h, N, D, device="cuda", generator=g).bfloat16() for h in (H, 1, 1, H))
    if args == "documents":
        ids = (torch.arange(N) // 1000).int()
        ids[150000:150100] = -1
        lo = (torch.arange(N) // 1000) * 1000
        lo[150100:151000] = 150100
        mask = fa.attention_mask(1, N, documents=ids[None].cuda())
    else:
        ids, lo = torch.zeros(N), torch.arange(N) - 899
        mask = fa.attention_mask(1, N, device="cuda", **args)
    o, lse = fa.attention_forward(q, k, v, mask=mask, softcap=cap)
    dq, dk, dv = fa.attention_backward(q, k, v, o, lse, do, mask=mask, softcap=cap)
    u, f = 2.0 ** -8, 2.0 ** -20
    for i in [0, 1, 127, 128, 899, 999, 1000, 131071, 150050, 150100, 150999, N - 1]:
        if ids[i] < 0:
            assert (o[0, :, i] == 0).all() and (dq[0, :, i] == 0).all() and (lse[0, :, i] == float("-inf")).all()
            continue
        a = max(0, int(lo[i]))
        kk, vv = k[0, 0, a:i + 1].double(), v[0, 0, a:i + 1].double()
        for h in range(H):
            s = kk @ q[0, h, i].double() / 8.0
            th = torch.tanh(s / cap)
            w = torch.softmax(cap * th, 0)
            e = f * (kk.abs() @ q[0, h, i].double().abs() / 8.0).max() + f * (1 + cap)
            want, L = w @ vv, torch.logsumexp(cap * th, 0)
            bound = (2 * e + f + u) * (w @ vv.abs()) + (u + f) * want.abs()
            assert abs(lse[0, h, i].double() - L) <= e + f * (1 + abs(L))
            assert ((o[0, h, i].double() - want).abs() <= bound).all()
            d = do[0, h, i].double()
            g1 = vv @ d - want @ d
            ds = w * (1 - th * th) * g1
            # dS: two roundings and P's error, and what delta takes from O's error
            dse = (2 * u + 4 * e + 2 * f) * ds.abs() + w * (f * (vv.abs() @ d.abs()) + (d.abs() * bound).sum()) * (1 + 2 * u)
            grad = ds @ kk / 8.0
            assert ((dq[0, h, i].double() - grad).abs() <= (dse + f * ds.abs()) @ kk.abs() / 8.0 + u * grad.abs()).all()
