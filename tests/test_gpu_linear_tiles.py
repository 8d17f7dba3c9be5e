"""Every kernel and tile shape of moe_linear with its whole epilogue, against the plain form in 64 bits.

FORMS names, for each type, the tile and tokens and rows that are sent to it: part tiles on both sides, and K that ends inside
a stage.  test_forms holds them to the rule, so that none of them can leave its kernel unseen.  Reference products are
formed in 64 bits on the GPU (the largest have 12.5 million results)."""
import pytest
import torch

import plain_ops as P
from routed_expert_ffn_layer_amd import moe

BF16, F32 = torch.bfloat16, torch.float32
SIZES = {(16, 4): (3, 77), (16, 8): (7, 77), (16, 16): (13, 77), (32, 32): (300, 523), (64, 32): (77, 4611), (64, 64): (61, 12301),
         (128, 64): (125, 12301), (128, 128): (250, 12301), (256, 128): (509, 12301), (256, 256): (1021, 12301)}
FORMS = [(dt, tile, *size) for dt in (BF16, F32) for tile, size in SIZES.items() if dt is BF16 or tile != (16, 8)]
TILES = [f for f in FORMS if f[1][0] > 16]
DEPTH = {BF16: 200, F32: 68}  # stages of 128 bytes and 16 bytes more
gpu = pytest.mark.gpu


@pytest.mark.parametrize("dt,tile,T,N", FORMS)
def test_forms(dt, tile, T, N):
    for K in (8, 64, DEPTH[dt], 520):
        assert moe.moe_linear_tile(moe.MOE_BF16 if dt is BF16 else moe.MOE_F32, T, N, K) == tile


def test_forms_of_invalid_shapes():
    for shape in ((moe.MOE_MXFP4, 4, 8, 64), (moe.MOE_BF16, 4, 8, 60), (moe.MOE_BF16, -1, 8, 64), (moe.MOE_BF16, 4, 0, 64), (moe.MOE_F32, 0, 8, 64)):
        assert moe.moe_linear_tile(*shape) == (0, 0)


def _wide(v, dt, pad):
    """v's rows pad columns apart, NaN between and behind them."""
    T, n = v.shape
    wide = torch.full((T + 1, n + pad), float("nan"), dtype=dt, device="cuda")
    wide[:T, :n] = v.to(dt)
    return wide[:T, :n]


def _untouched(y, pad):
    T, n = y.shape
    return torch.isnan(y._base[:, n:].float()).all() and torch.isnan(y._base[T:].float()).all() if pad else True


def _check(got, ref, tol):
    """P.check without the trip to the host."""
    got, fine = got.double(), torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    rest = ~fine & ~torch.isnan(ref)
    assert torch.equal(got[rest], ref[rest])
    bad = fine & ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i].item()!r} for {ref[i].item()!r}, "
                             f"bound {tol[i].item():.3g}")


def _operands(dt, T, N, K, seed, scale=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return n(T, K).to(dt), (scale * n(N, K)).to(dt), n(N), n(T, N)


@gpu
@pytest.mark.parametrize("act,bias,rdt,ydt,in_place,pad", [
    ("none", True, BF16, F32, False, 3), ("relu", True, None, BF16, False, 5), ("silu", False, F32, F32, True, 1),
    ("gelu", True, BF16, BF16, True, 0), ("gelu_tanh", True, F32, BF16, False, 8), ("none", False, None, BF16, False, 0)])
@pytest.mark.parametrize("dt,tile,T,N", FORMS)
def test_epilogue(dt, tile, T, N, act, bias, rdt, ydt, in_place, pad):
    """Bias, activation, residual of either type, in place too; operands, residual and result at strides of their own with
    NaN between their rows, which are neither read nor written."""
    x, w, b, r = _operands(dt, T, N, DEPTH[dt], T + N)
    b, r = b if bias else None, None if rdt is None else r.to(rdt)
    ref, tol = P.linear(x, w, b, act, r)
    y = _wide(torch.zeros(T, N) if not in_place else r, ydt, pad)
    res = None if r is None else y if in_place else _wide(r, rdt, 2 * pad + 1)
    apart = 8 if pad else 0
    moe.moe_linear(_wide(w, dt, 3 * apart), _wide(x, dt, apart), b, P.ACTS.index(act), res, y)
    torch.cuda.synchronize()
    _check(y, ref, P.stored(ref, tol, ydt))
    assert _untouched(y, pad)


@gpu
@pytest.mark.parametrize("K", [8, 56, 64, 72, 120, 128, 136, 192, 264, 520, 1032])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_depths_of_the_smallest_tile(K, dt):
    """Whole numbers, whose sums are exact: stages of 8 buffers, of which K fills from a part of one to several rounds."""
    T, N = 300, 523
    assert moe.moe_linear_tile(moe.MOE_BF16 if dt is BF16 else moe.MOE_F32, T, N, K) == (32, 32)
    g = torch.Generator(device="cuda").manual_seed(K)
    x, w = (torch.randint(-4, 5, (n, K), generator=g, device="cuda").to(dt) for n in (T, N))
    y = _wide(torch.zeros(T, N), F32, 3)
    moe.moe_linear(_wide(w, dt, 8), _wide(x, dt, 16), None, 0, None, y)
    torch.cuda.synchronize()
    assert torch.equal(y.double(), x.double() @ w.double().t()) and _untouched(y, 3)


@gpu
@pytest.mark.parametrize("dt,tile,T,N", TILES)
def test_columns_of_one_buffer(dt, tile, T, N):
    """x, the residual and the result side by side in the rows of one buffer."""
    K = DEPTH[dt]
    ld = (K + N + 8 + 7) // 8 * 8
    g = torch.Generator(device="cuda").manual_seed(T)
    buf = torch.randint(-4, 5, (T, ld), generator=g, device="cuda").to(dt)
    w = torch.randint(-2, 3, (N, K), generator=g, device="cuda").to(dt)
    before, at = buf.clone(), (K + 7) // 8 * 8
    moe.moe_linear(w, buf[:, :K], None, 0, buf[:, at:at + N], buf[:, at:at + N])
    torch.cuda.synchronize()
    ref = before[:, :K].double() @ w.double().t() + before[:, at:at + N].double()
    assert torch.equal(buf[:, at:at + N], ref.to(dt))  # whole numbers: the sum itself is exact
    assert torch.equal(buf[:, :at], before[:, :at]) and torch.equal(buf[:, at + N:], before[:, at + N:])


@gpu
@pytest.mark.parametrize("dt,tile,T,N", FORMS)
def test_infinities_and_nan_stay_in_their_rows(dt, tile, T, N):
    """In the last token, in the last weight row and in K's last elements, whose tiles and stages are not whole."""
    x, w, b, r = _operands(dt, T, N, DEPTH[dt], 5)
    x[T - 1, -1], w[N - 1, 0], r[0, 0], b[1] = float("inf"), float("nan"), float("inf"), float("-inf")
    y = torch.empty((T, N), device="cuda")
    moe.moe_linear(w, x, b, moe.MOE_ACT_RELU, r, y)
    torch.cuda.synchronize()
    ref, tol = P.linear(x, w, b, "relu", r)
    assert int(torch.isnan(ref).sum()) >= T and int(torch.isfinite(ref).sum()) > 0
    _check(y, ref, torch.nan_to_num(P.stored(ref, tol, F32), 0.0, 0.0, 0.0))


@gpu
@pytest.mark.parametrize("dt,tile,T,N", [f for f in TILES if f[1] in ((32, 32), (128, 64), (256, 256))])
def test_results_past_4_gib(dt, tile, T, N):
    """Rows of y, which is the residual too, up to 2^32 elements from its start."""
    buf = torch.empty(20 << 28, dtype=F32, device="cuda")
    y = buf.as_strided((T, N), ((buf.numel() - 16384) // (T - 1) // 8 * 8, 1))
    g = torch.Generator(device="cuda").manual_seed(T)
    x, w = (torch.randint(-4, 5, (n, 72), generator=g, device="cuda").to(dt) for n in (T, N))
    y.fill_(3.0)
    moe.moe_linear(w, x, None, 0, y, y)
    torch.cuda.synchronize()
    assert torch.equal(y.double(), x.double() @ w.double().t() + 3)
    del buf, y
    torch.cuda.empty_cache()
