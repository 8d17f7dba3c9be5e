"""Tokens sorted by expert and back, and the gradients, against their plain forms in 64 bits."""
import pytest
import torch

import plain_ops as P
from routed_expert_ffn_layer_amd import moe

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
MARK = 77.0  # what rows hold that no pair goes to


def _ids(T, k, E, seed, drop=0.0, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = (torch.randn(T, E, generator=g) - skew * torch.arange(E).float().log1p()).topk(k, 1).indices.to(torch.int32)
    bad = torch.rand(T, k, generator=g) < drop
    wrong = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=torch.int64)[torch.randint(0, 4, (T, k), generator=g)]
    return torch.where(bad, wrong, ids.long()).to(torch.int32)


def _wide(v, pad):
    wide = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=v.dtype, device="cuda")
    wide[:, :v.shape[1]] = v
    return wide[:, :v.shape[1]]


def _dispatch(x, ids, E, n_rows=None, pad=0):
    (T, k), H = ids.shape, x.shape[1]
    n_rows = T * k if n_rows is None else n_rows
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.full((n,), -7, **i32) for n in (E, E + 1, T * k, T * k)]
    rows = _wide(torch.full((n_rows, H), MARK, dtype=x.dtype), pad)
    ws = torch.empty(moe.moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda")
    moe.moe_dispatch(_wide(x, pad), ids.cuda(), E, *out, rows, ws)
    torch.cuda.synchronize()
    return [o.cpu() for o in out], rows


def _check_dispatch(T, k, E, H, dt, seed=0, drop=0.0, skew=0.0, n_rows=None, pad=0, ids=None):
    ids = _ids(T, k, E, seed, drop, skew) if ids is None else ids
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).to(dt)
    got, rows = _dispatch(x, ids, E, n_rows, pad)
    ref = P.order(ids, E)
    for name, a, b in zip(("counts", "offsets", "sorted_rows", "inv_rows"), got, ref):
        assert torch.equal(a, b), name
    want = torch.full(rows.shape, MARK, dtype=dt)
    n = min(int(ref[1][-1]), rows.shape[0])
    want[:n] = x[ref[2][:n].long() // k]
    assert torch.equal(rows.cpu(), want)
    if pad:
        assert torch.isnan(rows._base[:, H:].float()).all()


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (1, 32, 1024), (2, 1, 3), (16, 8, 256), (64, 6, 256), (128, 8, 60),
                                   (1024, 1, 1000), (1025, 1, 7), (129, 8, 256), (300, 6, 256), (1000, 8, 512), (4097, 6, 256),
                                   (3000, 32, 1024), (9000, 8, 128), (40000, 2, 1)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_order(T, k, E, drop):
    """One launch and three, one chunk round and several."""
    _check_dispatch(T, min(k, E), E, 24, BF16, seed=T, drop=drop, skew=1.1)


@pytest.mark.parametrize("H", [1, 2, 3, 7, 8, 9, 127, 512, 513, 520, 2048, 2049])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_rows(H, dt, pad):
    for T in (5, 700, 2100):
        _check_dispatch(T, 3, 9, H, dt, seed=H, pad=pad)


@pytest.mark.parametrize("T", [20, 900])
def test_no_pair_at_all_same_expert_twice_and_fewer_rows(T):
    _check_dispatch(T, 4, 16, 40, BF16, ids=torch.full((T, 4), -1, dtype=torch.int32))
    _check_dispatch(T, 4, 16, 40, BF16, ids=torch.full((T, 4), 15, dtype=torch.int32))
    _check_dispatch(T, 4, 16, 40, F32, n_rows=T, drop=0.1)
    _check_dispatch(T, 4, 16, 40, F32, n_rows=0)


def test_same_as_moe_permute():
    ids = _ids(500, 6, 256, 5, skew=1.1)
    got, _ = _dispatch(torch.zeros(500, 8), ids, 256)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.empty(n, **i32) for n in (256, 257, 3000, 3000)]  # 3000 pairs
    moe.moe_permute(ids.cuda(), 256, *out)
    torch.cuda.synchronize()
    for a, b in zip(got, out):
        assert torch.equal(a, b.cpu())


def test_no_tokens():
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets, none = torch.full((5,), -1, **i32), torch.full((6,), -1, **i32), torch.empty(0, **i32)
    moe.moe_dispatch(torch.empty((0, 8), device="cuda"), torch.empty((0, 2), **i32), 5, counts, offsets, none, none,
                     torch.empty((0, 8), device="cuda"))
    torch.cuda.synchronize()
    assert not counts.any() and not offsets.any()


def _state(T, k, E, H, dt, seed, drop=0.0):
    g = torch.Generator().manual_seed(seed + 1)
    ids = _ids(T, k, E, seed, drop)
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    rows = torch.randn(T * k, H, generator=g).to(dt)
    return ids, w, P.order(ids, E)[3], rows, g


@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (1, 8, 256, 2048), (3, 4, 8, 9), (16, 8, 64, 1000), (70, 5, 64, 513), (33, 32, 64, 100),
                                     (2500, 3, 8, 600)])
@pytest.mark.parametrize("rdt", [BF16, F32])
@pytest.mark.parametrize("ydt", [BF16, F32])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_combine_and_gradients(T, k, E, H, rdt, ydt, drop):
    ids, w, inv, rows, g = _state(T, k, E, H, rdt, T + H, drop)
    for pad, n_rows in ((0, T * k), (3, max(T * k - 2, 0))):
        r, at = _wide(rows, pad)[:n_rows], inv.cuda()
        y = _wide(torch.zeros(T, H, dtype=ydt), pad)
        moe.moe_combine_rows(r, w.cuda(), at, y)
        dx = _wide(torch.zeros(T, H, dtype=ydt), pad)
        moe.moe_dispatch_backward(r, at, k, dx)
        dy = torch.randn(T, H, generator=g).to(ydt)
        d_rows, d_w = _wide(torch.full((n_rows, H), MARK, dtype=rdt), pad), torch.full((T, k), MARK, device="cuda")
        moe.moe_combine_rows_backward(_wide(dy, pad), r, w.cuda(), at, d_rows, d_w)
        torch.cuda.synchronize()
        ref, mag = P.combine(rows, w, inv, T, n_rows)
        P.check(y, ref, P.stored(ref, k * P.U * mag, ydt), "y")  # k fused multiply-adds
        ref, mag = P.combine(rows, torch.ones(T, k), inv, T, n_rows)
        P.check(dx, ref, P.stored(ref, k * P.U * mag, ydt), "dx")
        live = (inv >= 0) & (inv < n_rows)
        pairs = torch.nonzero(live)[:, 0]
        place, tok = inv[pairs].long(), pairs // k
        ref, tol = torch.full((n_rows, H), MARK, dtype=torch.float64), torch.zeros(n_rows, H, dtype=torch.float64)
        ref[place] = w.reshape(-1)[pairs].double()[:, None] * dy.double()[tok]
        tol[place] = P.stored(ref[place], P.U * ref[place].abs(), rdt)
        P.check(d_rows, ref, tol, "d_rows")
        ref, mag = torch.zeros(T * k, dtype=torch.float64), torch.zeros(T * k, dtype=torch.float64)
        prod = dy.double()[tok] * rows.double()[place]
        ref[pairs], mag[pairs] = prod.sum(1), prod.abs().sum(1)
        P.check(d_w.reshape(-1), ref, H * P.U * mag, "d_w")  # H fused multiply-adds and additions at most


def test_rows_of_dropped_pairs_are_not_read():
    """A row that holds NaN, a weight that is NaN: of no effect where the pair is dropped."""
    rows, w = torch.randn(4, 40), torch.rand(2, 2)
    rows[3], w[1, 1] = float("nan"), float("nan")
    inv = torch.tensor([0, 2, 1, -1], dtype=torch.int32)
    y = torch.empty((2, 40), device="cuda")
    moe.moe_combine_rows(rows.cuda(), w.cuda(), inv.cuda(), y)
    torch.cuda.synchronize()
    w[1, 1] = 0.0
    ref, mag = P.combine(rows, w, inv, 2, 4)
    P.check(y, ref, P.stored(ref, 2 * P.U * mag, F32))


@pytest.mark.parametrize("T", [10, 2100])
def test_gradient_in_place_of_the_rows(T):
    ids, w, inv, rows, g = _state(T, 3, 7, 200, BF16, 4)
    dy, at, wd = torch.randn(T, 200, generator=g).to(BF16).cuda(), inv.cuda(), w.cuda()
    r = rows.cuda()
    want, dw, dw2 = torch.empty_like(r), torch.empty((T, 3), device="cuda"), torch.empty((T, 3), device="cuda")
    moe.moe_combine_rows_backward(dy, r, wd, at, want, dw)
    moe.moe_combine_rows_backward(dy, r, wd, at, r, dw2)
    torch.cuda.synchronize()
    assert torch.equal(want, r) and torch.equal(dw, dw2)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (5, 2, 63), (6, 3, 64), (7, 4, 65), (50, 32, 1024), (333, 6, 256)])
def test_gate(T, k, E):
    g = torch.Generator().manual_seed(T)
    ids = _ids(T, k, E, T, 0.2)
    w, dw = torch.softmax(torch.randn(T, k, generator=g), 1), torch.randn(T, k, generator=g)
    out = torch.full((T, E), MARK, device="cuda")
    moe.moe_gate_backward(ids.cuda(), w.cuda(), dw.cuda(), out)
    torch.cuda.synchronize()
    wd, d = w.double(), dw.double()
    ref, tol = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    grad = wd * (d - (wd * d).sum(1, keepdim=True))
    bound = (k + 4) * P.U * wd * (d.abs() + (wd * d).abs().sum(1, keepdim=True))
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if 0 <= e < E:
                ref[t, e] += grad[t, j]
                tol[t, e] += bound[t, j] * 2
    P.check(out, ref, tol)


def test_gate_of_one_expert_twice():
    ids = torch.tensor([[3, 3, 1]], dtype=torch.int32, device="cuda")
    w, d = torch.tensor([[0.5, 0.25, 0.25]], device="cuda"), torch.tensor([[1.0, 2.0, 4.0]], device="cuda")
    out = torch.empty((1, 5), device="cuda")
    moe.moe_gate_backward(ids, w, d, out)
    torch.cuda.synchronize()
    assert out.tolist() == [[0.0, 0.5, 0.0, -0.5, 0.0]]  # mean 2: w_j (d_j - 2) = -0.5, 0, 0.5


def test_gradients_against_differences():
    """Loss sum(dy y) of route -> dispatch -> an expert scaling its rows -> combine: the chain of the gradient
    calls against central differences of the plain form in 64 bits."""
    T, k, E, H = 6, 3, 8, 10
    g = torch.Generator().manual_seed(2)
    x, logits, dy = (torch.randn(*s, generator=g) for s in ((T, H), (T, E), (T, H)))
    scale = 1 + torch.rand(E, generator=g)
    ids = logits.topk(k, 1).indices.to(torch.int32)
    w = torch.softmax(logits.gather(1, ids.long()), 1)

    def loss(x, logits):
        w = torch.softmax(logits.gather(1, ids.long()), 1)
        return ((w * scale.double()[ids.long()])[..., None] * x[:, None, :] * dy.double()[:, None, :]).sum()

    (_, _, order, inv), rows = _dispatch(x, ids, E)
    expert = ids.reshape(-1)[order.long()].long()
    out = (rows.cpu() * scale[expert][:, None]).cuda()
    d_out, d_w = torch.empty_like(out), torch.empty((T, k), device="cuda")
    moe.moe_combine_rows_backward(dy.cuda(), out, w.cuda(), inv.cuda(), d_out, d_w)
    d_in = (d_out.cpu() * scale[expert][:, None]).cuda()
    dx, d_logits = torch.empty((T, H), device="cuda"), torch.empty((T, E), device="cuda")
    moe.moe_dispatch_backward(d_in, inv.cuda(), k, dx)
    moe.moe_gate_backward(ids.cuda(), w.cuda(), d_w, d_logits)
    torch.cuda.synchronize()
    h = 1e-5
    for got, at in ((dx, 0), (d_logits, 1)):
        args = [x.double(), logits.double()]
        diff = torch.zeros_like(args[at])
        for i in range(diff.numel()):
            hi, lo = [a.clone() for a in args], [a.clone() for a in args]
            hi[at].view(-1)[i] += h
            lo[at].view(-1)[i] -= h
            diff.view(-1)[i] = (loss(*hi) - loss(*lo)) / (2 * h)
        # f32 chain: sums of up to H k terms of size about 10; differences: 64-bit roundings over h and h^2
        P.check(got, diff, 200 * P.U * 10 + 1e-8)


def test_same_bits_and_graph():
    """All six calls captured together, replayed on new inputs with eager work between."""
    T, k, E, H = 600, 4, 32, 264
    g = torch.Generator().manual_seed(8)
    ids, x = _ids(T, k, E, 1).cuda(), torch.randn(T, H, generator=g).to(BF16).cuda()
    w, dy = torch.softmax(torch.randn(T, k, generator=g), 1).cuda(), torch.randn(T, H, generator=g).to(BF16).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")

    def buffers():
        return dict(order=[torch.zeros(n, **i32) for n in (E, E + 1, T * k, T * k)], rows=torch.zeros((T * k, H), dtype=BF16, device="cuda"),
                    ws=torch.empty(moe.moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda"), y=torch.zeros_like(x),
                    d_rows=torch.zeros((T * k, H), dtype=BF16, device="cuda"), d_w=torch.zeros_like(w), dx=torch.zeros_like(x),
                    dl=torch.zeros((T, E), device="cuda"))

    def step(b):
        moe.moe_dispatch(x, ids, E, *b["order"], b["rows"], b["ws"])
        moe.moe_combine_rows(b["rows"], w, b["order"][3], b["y"])
        moe.moe_combine_rows_backward(dy, b["rows"], w, b["order"][3], b["d_rows"], b["d_w"])
        moe.moe_dispatch_backward(b["d_rows"], b["order"][3], k, b["dx"])
        moe.moe_gate_backward(ids, w, b["d_w"], b["dl"])

    flat = lambda b: b["order"] + [b[n] for n in ("rows", "y", "d_rows", "d_w", "dx", "dl")]  # noqa: E731
    one, two = buffers(), buffers()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step(one)
    for i in range(3):
        x.mul_(-1.5)
        ids.copy_((ids + 1) % E)
        step(two)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(flat(one), flat(two)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [60, 600, 5000])
def test_two_streams_at_once(T):
    """The way there and back of different tokens on two streams, each with its tables and workspace."""
    k, E, H, jobs = 6, 64, 512, []
    for seed in range(2):
        ids, x = _ids(T, k, E, seed), torch.randn(T, H, generator=torch.Generator().manual_seed(seed))
        w = torch.rand(T, k, generator=torch.Generator().manual_seed(seed))
        i32 = dict(dtype=torch.int32, device="cuda")
        out = [torch.full((n,), -7, **i32) for n in (E, E + 1, T * k, T * k)]
        ws = torch.empty(moe.moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda")
        jobs.append((torch.cuda.Stream(), x.cuda(), ids.cuda(), w.cuda(), out, torch.zeros((T * k, H), device="cuda"),
                     torch.zeros((T, H), device="cuda"), ws, P.order(ids, E)))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, x, ids, w, out, rows, y, ws, _ in jobs:
            moe.moe_dispatch(x, ids, E, *out, rows, ws, stream=st)
            moe.moe_combine_rows(rows, w, out[3], y, stream=st)
    torch.cuda.synchronize()
    for _, x, ids, w, out, rows, y, ws, ref in jobs:
        for a, b in zip(out, ref):
            assert torch.equal(a.cpu(), b)
        assert torch.equal(rows.cpu(), x.cpu()[ref[2].long() // k])
        want = x.cpu().double() * w.cpu().double().sum(1, keepdim=True)  # every pair brings its token's own row back
        bound = (k + 1) * 2.0 ** -24 * 1.01 * want.abs() + 2.0 ** -126  # k products and sums, one store
        assert ((y.cpu().double() - want).abs() <= bound).all()
