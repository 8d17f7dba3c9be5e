"""moe_linear against its plain form in 64 bits: integers, whose sums are exact, for equality over the
shapes, real numbers for the epilogue."""
import pytest
import torch

import plain_ops as P
from routed_expert_ffn_layer_amd import moe

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _wide(v, dt, pad):
    """v's rows pad columns apart, NaN between and behind them."""
    T, n = v.shape
    wide = torch.full((T + 1, n + pad), float("nan"), dtype=dt, device="cuda")
    wide[:T, :n] = v.to(dt)
    return wide[:T, :n]


def _integers(dt, T, N, K, seed=0, xpad=0, wpad=0, ypad=0, most=4):
    """Sums of products of integers up to `most`: under 2^24 and so exact in any order."""
    assert most * most * K < 1 << 24
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + N * 17 + K)
    x = torch.randint(-most, most + 1, (T, K), generator=g).double()
    w = torch.randint(-most, most + 1, (N, K), generator=g).double()
    y = _wide(torch.zeros(T, N), F32, ypad)
    moe.moe_linear(_wide(w, dt, wpad), _wide(x, dt, xpad), None, moe.MOE_ACT_NONE, None, y)
    torch.cuda.synchronize()
    ref = x @ w.t()
    assert torch.equal(y.cpu().double(), ref), f"{int((y.cpu().double() != ref).sum())} of {ref.numel()} differ"
    if ypad:
        assert torch.isnan(y._base[:, N:]).all() and torch.isnan(y._base[T:]).all()


@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 513])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_tokens(T, dt):
    _integers(dt, T, 200, 136)
    _integers(dt, T, 256, 512)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 256, 257, 1003])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_rows(N, dt):
    for T in (1, 20, 70, 300):
        _integers(dt, T, N, 264)


@pytest.mark.parametrize("K", [8, 16, 24, 32, 40, 56, 64, 72, 120, 128, 136, 192, 248, 256, 264, 512, 520, 1024, 2088, 4096, 8200])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_depths(K, dt):
    for T in (3, 18, 66, 260):
        _integers(dt, T, 48, K)


@pytest.mark.parametrize("K", [4, 12, 20, 36, 60, 68, 132])
def test_depths_of_f32(K):
    for T in (3, 40, 100):
        _integers(F32, T, 33, K)


@pytest.mark.parametrize("T,N,K", [(300, 520, 328), (520, 300, 64), (1024, 512, 1024), (777, 1300, 200), (2048, 2304, 136), (1000, 4000, 88)])
def test_many_tokens(T, N, K):
    _integers(BF16, T, N, K)


@pytest.mark.parametrize("T", [19, 61, 125, 250, 509, 1021])
@pytest.mark.parametrize("K", [8, 72, 128, 520, 1032])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_tile_shapes(T, K, dt):
    """Every tile shape with part tiles on both sides and part stages: the more tokens, the larger the tile
    whose number over 12301 rows comes closest to that of the CUs."""
    _integers(dt, T, 12301, K)


@pytest.mark.parametrize("T", [5, 30, 90, 400])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_strides(T, dt):
    """Rows apart from each other, NaN between them: nothing of it is read into a sum or written."""
    _integers(dt, T, 77, 200, xpad=8, wpad=24, ypad=3)
    _integers(dt, T, 128, 128, xpad=64, wpad=8, ypad=1)


@pytest.mark.parametrize("T", [1, 24, 130, 600])
@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("dt,rdt,ydt", [(BF16, BF16, BF16), (BF16, F32, F32), (F32, F32, F32), (F32, BF16, BF16), (BF16, F32, BF16)])
def test_epilogue(T, act, dt, rdt, ydt):
    g = torch.Generator().manual_seed(act + T)
    N, K = 150, 96
    x, w = torch.randn(T, K, generator=g).to(dt), (torch.randn(N, K, generator=g) * 0.2).to(dt)
    bias, res = torch.randn(N, generator=g), torch.randn(T, N, generator=g).to(rdt)
    for b, r in ((bias, res), (None, res), (bias, None), (None, None)):
        y = torch.full((T, N), float("nan"), dtype=ydt, device="cuda")
        moe.moe_linear(w.cuda(), x.cuda(), None if b is None else b.cuda(), act, None if r is None else r.cuda(), y)
        torch.cuda.synchronize()
        ref, tol = P.linear(x, w, b, P.ACTS[act], r)
        P.check(y, ref, P.stored(ref, tol, ydt), f"bias {b is not None}, res {r is not None}")


@pytest.mark.parametrize("act", range(5))
def test_activation_range(act):
    """Values from far below to far above 0: identity weights pass x to the activation."""
    v = torch.cat([torch.linspace(-30, 30, 481), torch.tensor([0.0, 1e-20, -1e-20, 100.0, -100.0, 3e4, -3e4])]).to(BF16).float()
    v = torch.cat([v, torch.zeros(-len(v) % 8)])
    x = torch.diag(v).to(BF16)
    y = torch.empty((len(v), 8), device="cuda")
    w = torch.ones((8, len(v)), dtype=BF16)
    moe.moe_linear(w.cuda(), x.cuda(), None, act, None, y)
    torch.cuda.synchronize()
    ref = P.act(v.double(), P.ACTS[act])[:, None].expand(-1, 8)
    tol = P.act_bound(v.double(), torch.zeros(len(v), dtype=torch.float64), P.ACTS[act])[:, None]
    P.check(y, ref, P.stored(ref, tol, F32))


@pytest.mark.parametrize("T", [2, 40, 300])
def test_residual_in_place(T):
    g = torch.Generator().manual_seed(T)
    x, w = torch.randn(T, 64, generator=g).to(BF16).cuda(), torch.randn(90, 64, generator=g).to(BF16).cuda()
    res = torch.randn(T, 90, generator=g).to(BF16).cuda()
    want = torch.empty_like(res)
    moe.moe_linear(w, x, None, moe.MOE_ACT_SILU, res, want)
    moe.moe_linear(w, x, None, moe.MOE_ACT_SILU, res, res)
    torch.cuda.synchronize()
    assert torch.equal(want, res)


@pytest.mark.parametrize("T", [1, 20, 100, 300])
def test_infinities_and_nan_stay_in_their_rows(T):
    g = torch.Generator().manual_seed(T)
    x, w = torch.randn(T, 72, generator=g), torch.randn(40, 72, generator=g)
    x[T - 1, 71] = float("inf")
    w[39, 0] = float("nan")
    y = torch.empty((T, 40), device="cuda")
    moe.moe_linear(w.to(BF16).cuda(), x.to(BF16).cuda(), None, 0, None, y)
    torch.cuda.synchronize()
    ref, tol = P.linear(x.to(BF16), w.to(BF16), None, "none", None)
    P.check(y, ref, torch.nan_to_num(P.stored(ref, tol, F32), 0.0, 0.0, 0.0))


@pytest.mark.parametrize("T", [1, 64, 500])
def test_same_bits_and_other_stream_and_graph(T):
    g = torch.Generator().manual_seed(T)
    x, w = torch.randn(T, 2048, generator=g).to(BF16).cuda(), torch.randn(600, 2048, generator=g).to(BF16).cuda()
    want, y = torch.empty((T, 600), device="cuda"), torch.zeros((T, 600), device="cuda")
    moe.moe_linear(w, x, None, 0, None, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        moe.moe_linear(w, x, None, 0, None, y)
        side.synchronize()
        assert torch.equal(y, want)
        with torch.cuda.graph(graph, stream=side):
            moe.moe_linear(w, x, None, 0, None, y)
    for i in range(3):
        x.mul_(-0.5)
        moe.moe_linear(w, x, None, 0, None, want)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_no_tokens():
    moe.moe_linear(torch.zeros((8, 8), device="cuda"), torch.zeros((0, 8), device="cuda"), None, 0, None, torch.zeros((0, 8), device="cuda"))


@pytest.mark.parametrize("T", [3, 50, 300])
def test_columns_of_one_buffer(T):
    """x, the residual and the result side by side in the rows of one buffer: nothing overlaps."""
    g = torch.Generator().manual_seed(T)
    buf = torch.randint(-4, 5, (T, 64 + 24 + 40), generator=g).to(BF16)
    w = torch.randint(-2, 3, (40, 64), generator=g).to(BF16)
    d = buf.cuda()
    moe.moe_linear(w.cuda(), d[:, :64], None, 0, d[:, 88:], d[:, 88:])
    torch.cuda.synchronize()
    ref = buf.double()[:, :64] @ w.double().t() + buf.double()[:, 88:]
    assert torch.equal(d[:, :88].cpu(), buf[:, :88])
    assert torch.equal(d[:, 88:].cpu(), ref.to(BF16))  # integers past 256 are rounded, the sum itself is exact


def test_two_streams_at_once():
    """Different products on two streams, many times over: each as alone."""
    g = torch.Generator().manual_seed(1)
    jobs = []
    for T, N, K in ((300, 700, 1024), (16, 5000, 512)):
        x, w = torch.randn(T, K, generator=g).to(BF16).cuda(), torch.randn(N, K, generator=g).to(BF16).cuda()
        want, y = torch.empty((T, N), device="cuda"), torch.zeros((T, N), device="cuda")
        moe.moe_linear(w, x, None, 0, None, want)
        jobs.append((torch.cuda.Stream(), w, x, y, want))
    torch.cuda.synchronize()
    for _ in range(50):
        for st, w, x, y, _ in jobs:
            moe.moe_linear(w, x, None, 0, None, y, stream=st)
    torch.cuda.synchronize()
    for _, _, _, y, want in jobs:
        assert torch.equal(y, want)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("K", [8, 120, 128, 136, 264, 2040, 4104])
def test_small_results_exactly(dt, K):
    """Whole numbers, whose sums are exact: every form for few tokens or small results, rows and K that end inside its tiles and
    steps, and nothing written outside y."""
    g = torch.Generator().manual_seed(K)
    X, W = torch.randint(-3, 4, (70, K), generator=g).double(), torch.randint(-3, 4, (300, K), generator=g).double()
    x, w, ref = X.to(dt).cuda(), W.to(dt).cuda(), X @ W.t()
    for T in (1, 2, 3, 4, 5, 7, 8, 9, 12, 15, 16, 17, 31, 33, 70):
        for N in (1, 7, 15, 16, 17, 40, 300):
            y = torch.full((T + 1, N + 3), 77.0, device="cuda")
            moe.moe_linear(w[:N], x[:T], None, 0, None, y[:T, :N])
            got = y.cpu().double()
            assert torch.equal(got[:T, :N], ref[:T, :N]), (T, N)
            assert (got[T] == 77).all() and (got[:, N:] == 77).all(), (T, N)
