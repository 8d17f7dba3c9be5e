"""The linear product with 4-bit weights (moe_w4_pack, moe_w4_linear) against the
definition in 64 bits, and a decode step of products, router and experts together.

Bound.  Operands are exact (the integer codes, E2M1 times a power of two and bf16
activations), so only the f32 sums round, u = 2^-24 each: a sum of K products in any
order is off by at most 2 (K + 64) u times the sum of magnitudes (the factor 2: a matrix
instruction's own sum need not round to nearest).  For INT4 the magnitudes are those of
s (q |x| + z |x|), as the group's sums of x q and of x are formed apart; each group adds
three roundings, 3 ceil(K/G) <= K in all: 2 (2 K + 64) u.  A bf16 output adds half a step,
2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import synth
from helpers import dev, log, to_dev
from routed_expert_ffn_layer_amd import layer as L
from routed_expert_ffn_layer_amd import moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def _weights(fmt, N, K, group, seed, zeros=True):
    g = np.random.default_rng(seed)
    codes = g.integers(0, 256, (N, K // 2), dtype=np.uint8)
    n = -(-K // group)
    if fmt == moe.MOE_MXFP4:
        return codes, g.integers(110, 130, (N, n), dtype=np.uint8), None
    scales = (g.random((N, n)) * 0.02 - 0.005).astype(np.float16)
    return codes, scales, g.integers(0, 16, (N, n), dtype=np.uint8) if zeros else None


def _dequant(fmt, codes, scales, zeros, K, group):
    """W and the magnitudes its sums run over, float64 [N][K]."""
    q = np.empty((codes.shape[0], K), np.int64)
    q[:, 0::2], q[:, 1::2] = codes & 15, codes >> 4
    per = np.repeat(scales, group, axis=1)[:, :K]
    if fmt == moe.MOE_MXFP4:
        w = E2M1[q] * np.exp2(per.astype(np.float64) - 127)
        return w, np.abs(w)
    z = np.full_like(q, 8) if zeros is None else np.repeat(zeros, group, axis=1)[:, :K].astype(np.int64)
    return (q - z) * per.astype(np.float64), (q + z) * np.abs(per.astype(np.float64))


def _x(T, K, seed):
    return synth.bf16_bits(np.random.default_rng(seed).standard_normal((T, K)).astype(np.float32))


def _pack(fmt, codes, scales, zeros, K, group):
    N = codes.shape[0]
    w = torch.full((moe.moe_w4_bytes(fmt, N, K, group) + 64,), 0xA5, dtype=torch.uint8, device=dev())
    moe.moe_w4_pack(fmt, to_dev(codes), to_dev(scales), None if zeros is None else to_dev(zeros), N, K, group, w)
    assert bool((w[-64:] == 0xA5).all())
    return w


def _check(got, w, mag, x, bias, bf16, what):
    xf = synth.bf16_bits_to_f32(x).astype(np.float64)
    ref = xf @ w.T
    K = w.shape[1]
    lim = 2 * (2 * K + 64) * U * (np.abs(xf) @ mag.T) + 1e-37
    if bias is not None:
        ref = ref + bias.astype(np.float64)
        lim = lim + U * np.abs(ref)
    if bf16:
        lim = lim + 1.01 * 2.0 ** -8 * np.abs(ref)
    err = np.abs(got.double().cpu().numpy() - ref)
    worst = float(np.max(err / lim)) if ref.size else 0.0
    log(f"{what}: error / bound = {worst:.3f}")
    assert worst <= 1.0, what


FORMATS = [(moe.MOE_MXFP4, 32), (moe.MOE_INT4, 32), (moe.MOE_INT4, 64), (moe.MOE_INT4, 128)]
SHAPES = [
    # T, N, K, bias, bf16 output
    (1, 16, 128, False, False),
    (1, 1, 32, True, False),          # the smallest
    (2, 15, 96, False, True),
    (3, 17, 160, True, False),        # one row past a tile, a column step of 32
    (4, 1003, 2080, False, False),    # a partial last group of 64 and 128
    (5, 512, 4096, True, True),
    (8, 40, 1024, False, False),
    (9, 250, 224, False, True),
    (16, 100, 640, True, False),
    (17, 33, 2176, False, False),
    (33, 64, 96, False, False),
    (64, 300, 1056, True, True),
    (65, 48, 256, False, False),
    (130, 31, 288, True, False),
    (1, 20000, 512, False, True),
    (7, 9000, 8192, False, False),
    (64, 5000, 4096, False, False),   # blocks of 4 row tiles
    (20, 9000, 416, True, True),
    (20, 45003, 256, False, False),   # blocks of 16
    (64, 45003, 160, True, True),
    (70, 45000, 288, False, False),   # and a second pass of 6 tokens
    (1, 200, 8192, False, False),     # two chunks of steps per wave
    (16, 100, 6112, False, True),
    (3, 64, 9024, True, False),       # more than two
    (6, 40, 9024, False, False),
    (12, 33, 16384, False, False),
]


@pytest.mark.parametrize("fmt,group", FORMATS, ids=["mxfp4", "int4_32", "int4_64", "int4_128"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "_".join(str(int(v)) for v in s))
def test_product_against_64_bits(fmt, group, shape):
    T, N, K, with_bias, bf16 = shape
    log(f"w4 fmt={fmt} group={group} {shape}")
    codes, scales, zeros = _weights(fmt, N, K, group, seed=N + K)
    x = _x(T, K, T)
    bias = np.random.default_rng(1).standard_normal(N).astype(np.float32) if with_bias else None
    w = _pack(fmt, codes, scales, zeros, K, group)
    y = torch.empty((T, N), dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
    moe.moe_w4_linear(fmt, w, N, K, group, to_dev(x), None if bias is None else to_dev(bias), y)
    torch.cuda.synchronize()
    _check(y, *_dequant(fmt, codes, scales, zeros, K, group), x, bias, bf16, f"{fmt} {group} {shape}")


@pytest.mark.parametrize("fmt,group", FORMATS, ids=["mxfp4", "int4_32", "int4_64", "int4_128"])
@pytest.mark.parametrize("T", [3, 40])
def test_row_strides_and_what_lies_around(fmt, group, T):
    """x a slice of wider rows that hold NaN beside it, y a slice of a wider tensor."""
    N, K = 77, 1120
    codes, scales, zeros = _weights(fmt, N, K, group, seed=5)
    x = _x(T, K, 6)
    wide = torch.full((T + 1, K + 24), float("nan"), dtype=torch.bfloat16, device=dev())
    wide[:T, 8:8 + K] = to_dev(x).view(torch.bfloat16)
    out = torch.full((T + 2, N + 51), 7.0, device=dev())
    w = _pack(fmt, codes, scales, zeros, K, group)
    y = out[:T, 4:4 + N]
    moe.moe_w4_linear(fmt, w, N, K, group, wide[:T, 8:8 + K], None, y)
    torch.cuda.synchronize()
    _check(y, *_dequant(fmt, codes, scales, zeros, K, group), x, None, False, "strided")
    y.fill_(7.0)
    assert bool((out == 7.0).all())


def test_default_zero_is_8():
    N, K = 48, 384
    codes, scales, _ = _weights(moe.MOE_INT4, N, K, 128, seed=2, zeros=False)
    x = _x(5, K, 3)
    ys = []
    for z in (None, np.full(scales.shape, 8, np.uint8)):
        y = torch.empty((5, N), device=dev())
        moe.moe_w4_linear(moe.MOE_INT4, _pack(moe.MOE_INT4, codes, scales, z, K, 128), N, K, 128, to_dev(x), None, y)
        ys.append(y)
    assert torch.equal(*ys)
    _check(ys[0], *_dequant(moe.MOE_INT4, codes, scales, None, K, 128), x, None, False, "zero 8")


def test_extreme_scales_and_zeros():
    """f16 scales of zero, the least subnormal and the largest; zeros up to 255; E8M0
    scales from 2^-127 (a subnormal factor) up, one block NaN."""
    K, N = 256, 32
    codes, scales, zeros = _weights(moe.MOE_INT4, N, K, 64, seed=11)
    scales[0], scales[1], scales[2] = 0, np.float16(6e-8), np.float16(65504)
    zeros[3], zeros[4] = 255, 0
    x = _x(4, K, 12)
    y = torch.empty((4, N), device=dev())
    moe.moe_w4_linear(moe.MOE_INT4, _pack(moe.MOE_INT4, codes, scales, zeros, K, 64), N, K, 64, to_dev(x), None, y)
    _check(y, *_dequant(moe.MOE_INT4, codes, scales, zeros, K, 64), x, None, False, "int4 extremes")
    assert bool((y[:, 0] == 0).all())
    codes, scales, _ = _weights(moe.MOE_MXFP4, N, K, 32, seed=13)
    scales[0], scales[1], scales[2, 0] = 0, 1, 255
    codes[0, :] |= 0x22  # no zeros: codes of at least 1.0
    y = torch.empty((4, N), device=dev())
    moe.moe_w4_linear(moe.MOE_MXFP4, _pack(moe.MOE_MXFP4, codes, scales, None, K, 32), N, K, 32, to_dev(x), None, y)
    assert bool(torch.isnan(y[:, 2]).all())
    keep = np.arange(N) != 2
    w, mag = _dequant(moe.MOE_MXFP4, codes[keep], scales[keep], None, K, 32)
    # products with bf16 subnormals may flush: each is off by at most 2^-126 |x|
    xf = np.abs(synth.bf16_bits_to_f32(x).astype(np.float64))
    ref = synth.bf16_bits_to_f32(x).astype(np.float64) @ w.T
    lim = 2 * (2 * K + 64) * U * (xf @ mag.T) + 2.0 ** -126 * (K + xf.sum(1, keepdims=True))
    assert np.all(np.abs(y.double().cpu().numpy()[:, keep] - ref) <= lim)


@pytest.mark.parametrize("fmt,group", FORMATS, ids=["mxfp4", "int4_32", "int4_64", "int4_128"])
@pytest.mark.parametrize("T,N", [(20, 9000), (64, 5000), (40, 33000)])
@pytest.mark.parametrize("K", [32, 288])
def test_an_odd_number_of_column_steps(T, N, K, fmt, group):
    """Blocks of 4 and 16 row tiles whose last pair of column steps has one: close to the formula, and a
    token with infinities and NaN in that step stays its own."""
    codes, scales, zeros = _weights(fmt, N, K, group, seed=61)
    w = _pack(fmt, codes, scales, zeros, K, group)
    xb = _x(T, K, 62)
    x = to_dev(xb).view(torch.bfloat16)
    y, y2 = torch.empty((T, N), device=dev()), torch.empty((T, N), device=dev())
    moe.moe_w4_linear(fmt, w, N, K, group, x, None, y)
    _check(y, *_dequant(fmt, codes, scales, zeros, K, group), xb, None, False, f"{fmt} {group} {T} {N} {K}")
    x[3, K - 1], x[T - 1, K - 2] = float("inf"), float("nan")
    moe.moe_w4_linear(fmt, w, N, K, group, x, None, y2)
    keep = [t for t in range(T) if t not in (3, T - 1)]
    assert torch.equal(y[keep], y2[keep]) and bool(torch.isnan(y2[T - 1]).all())


def test_a_bad_token_stays_its_own():
    for fmt, group in FORMATS:
        N, K = 40, 512
        codes, scales, zeros = _weights(fmt, N, K, group, seed=21)
        w = _pack(fmt, codes, scales, zeros, K, group)
        x = to_dev(_x(20, K, 22)).view(torch.bfloat16)
        y, y2 = torch.empty((20, N), device=dev()), torch.empty((20, N), device=dev())
        moe.moe_w4_linear(fmt, w, N, K, group, x, None, y)
        x[3, 500], x[17, 0] = float("inf"), float("nan")
        moe.moe_w4_linear(fmt, w, N, K, group, x, None, y2)
        keep = [t for t in range(20) if t not in (3, 17)]
        assert torch.equal(y[keep], y2[keep]) and bool(torch.isnan(y2[17]).all())


@pytest.mark.parametrize("fmt,group", [(moe.MOE_MXFP4, 32), (moe.MOE_INT4, 128)])
def test_codes_past_4_gib(fmt, group):
    """A matrix of more than 2^32 bytes of codes; rows at both ends and across the border."""
    N, K, T = 70000, 131072, 2
    g = torch.Generator(device=dev()).manual_seed(3)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=dev(), generator=g)
    n = K // group
    if fmt == moe.MOE_MXFP4:
        scales, zeros = torch.randint(115, 125, (N, n), dtype=torch.uint8, device=dev(), generator=g), None
    else:
        scales = (torch.rand((N, n), device=dev(), generator=g) * 0.01).to(torch.float16)
        zeros = torch.randint(0, 16, (N, n), dtype=torch.uint8, device=dev(), generator=g)
    w = torch.empty(moe.moe_w4_bytes(fmt, N, K, group), dtype=torch.uint8, device=dev())
    moe.moe_w4_pack(fmt, codes, scales, zeros, N, K, group, w)
    x = _x(T, K, 4)
    y = torch.empty((T, N), device=dev())
    moe.moe_w4_linear(fmt, w, N, K, group, to_dev(x), None, y)
    torch.cuda.synchronize()
    border = 2 ** 32 // (K // 2)
    rows = [0, 1, 17, border - 16, border - 1, border, border + 1, border + 15, N - 17, N - 1]
    take = lambda t: t[rows].cpu().numpy()
    wr, mag = _dequant(fmt, take(codes), take(scales), None if zeros is None else take(zeros), K, group)
    _check(y[:, rows], wr, mag, x, None, False, "past 4 GiB")


@pytest.mark.parametrize("fmt,group", [(moe.MOE_MXFP4, 32), (moe.MOE_INT4, 64)])
@pytest.mark.parametrize("T", [1, 30])
def test_replays_and_streams(fmt, group, T):
    N, K = 515, 2048
    codes, scales, zeros = _weights(fmt, N, K, group, seed=51)
    w = _pack(fmt, codes, scales, zeros, K, group)
    xs = [to_dev(_x(T, K, 60 + i)) for i in range(3)]

    def eager(x, stream=None):
        y = torch.empty((T, N), dtype=torch.bfloat16, device=dev())
        moe.moe_w4_linear(fmt, w, N, K, group, x, None, y, stream)
        return y

    refs = [eager(x) for x in xs]
    x_s, y_s = xs[0].clone(), torch.empty((T, N), dtype=torch.bfloat16, device=dev())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_w4_linear(fmt, w, N, K, group, x_s, None, y_s)
    for rep in range(4):
        x_s.copy_(xs[rep % 3])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y_s, refs[rep % 3])
        assert torch.equal(eager(xs[(rep + 1) % 3]), refs[(rep + 1) % 3])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = eager(xs[1], s1), eager(xs[2], s2)
    torch.cuda.synchronize()
    assert torch.equal(a, refs[1]) and torch.equal(b, refs[2])


def test_refusals_of_the_binding():
    """Shapes, strides and devices that the C entry cannot see."""
    N, K = 32, 64
    w = torch.zeros(moe.moe_w4_bytes(moe.MOE_INT4, N, K, 64), dtype=torch.uint8, device=dev())
    x, y = torch.zeros((3, K), dtype=torch.bfloat16, device=dev()), torch.zeros((3, N), device=dev())
    call = lambda x, y, w=w: moe.moe_w4_linear(moe.MOE_INT4, w, N, K, 64, x, None, y)
    call(x, y)
    for bx, by, bw in ((x[:, :32], y, w), (x, y[:2], w), (x, y[:, :16], w), (x, y.double(), w), (x.cpu(), y, w), (x, y, w.cpu()),
                       (torch.zeros((K, 3), dtype=torch.bfloat16, device=dev()).t(), y, w),
                       (x, torch.zeros((N, 3), device=dev()).t(), w)):
        with pytest.raises(moe.MoeError) as e:
            call(bx, by, bw)
        assert e.value.status == moe.MOE_EINVAL
    with pytest.raises(moe.MoeError) as e:
        moe.moe_w4_pack(moe.MOE_INT4, w, w, None, N, K, 64, w[:-1])
    assert e.value.status == moe.MOE_ECAPACITY


@pytest.mark.parametrize("fmt,group", [(moe.MOE_MXFP4, 32), (moe.MOE_INT4, 128)])
def test_a_decode_step_together(ora, fmt, group):
    """Projection with 4-bit weights, router logits with 4-bit weights, the layer on them, and
    a head over a small vocabulary: each step against 64 bits on what it was handed."""
    from test_gpu_layer_decode import _check as check_layer, _reference
    T, H, I, E, k, V = 6, 256, 64, 24, 4, 500
    mats = {n: _weights(fmt, rows, H, group, seed=70 + rows) for n, rows in (("in", H), ("router", E), ("head", V))}
    packed = {n: _pack(fmt, *m, H, group) for n, m in mats.items()}
    x0 = _x(T, H, 71)
    lay = synth.small_layer(synth.MXFP4, T, H, I, E, k, seed=72, shared=True, I_shared=32)
    experts, shared = to_dev(lay["experts"]), to_dev(lay["shared"])
    x = torch.empty((T, H), dtype=torch.bfloat16, device=dev())
    logits, out = torch.empty((T, E), device=dev()), torch.empty((T, V), device=dev())
    b = L.LayerBuffers(T, E, k, H, I, moe.MOE_MXFP4, I_shared=32)
    moe.moe_w4_linear(fmt, packed["in"], H, H, group, to_dev(x0), None, x)
    moe.moe_w4_linear(fmt, packed["router"], E, H, group, x, None, logits)
    y = L.forward_decode(b, logits, x, experts, experts.shape[1], L.identity_slots(E), shared)
    moe.moe_w4_linear(fmt, packed["head"], V, H, group, y, None, out)
    torch.cuda.synchronize()
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)
    _check(x, *_dequant(fmt, *mats["in"], H, group), x0, None, True, "projection")
    _check(logits, *_dequant(fmt, *mats["router"], H, group), bits(x), None, False, "router")
    lay["x"], lay["logits"] = bits(x), logits.cpu().numpy()
    ids, _, w64 = ora.route_topk(lay["logits"], k)
    np.testing.assert_array_equal(b.topk_ids.cpu().numpy(), ids)
    ref, bound = _reference(ora, lay, ids, w64)
    check_layer(y, ref, bound, True, "layer")
    _check(out, *_dequant(fmt, *mats["head"], H, group), bits(y), None, False, "head")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K", [(1, 40, 512), (4, 33, 9024), (3, 50, 8192), (7, 40, 512), (8, 20, 6112), (6, 40, 9024),
                                   (16, 40, 544), (12, 33, 6112), (9, 17, 16384), (17, 40, 512), (20, 9000, 416),
                                   (64, 5000, 256), (40, 33000, 96), (30, 45003, 96), (70, 45000, 160)])
def test_infinite_and_huge_activations(T, N, K, group):
    """INT4 holds y = sum s (q - z) x over every x: an infinite x gives the infinity of its products'
    sign, NaN only where q = z (or two infinities differ), and finite x whose sums with the codes alone would
    pass the f32 range give the finite result.  The weights are small enough that no sum of whole products
    does.  With K such products the bound of the module holds, its magnitudes included."""
    codes, scales, zeros = _weights(moe.MOE_INT4, N, K, group, seed=81)
    zeros[::3] = np.random.default_rng(82).integers(0, 256, zeros[::3].shape)
    scales[scales == 0] = np.float16(0.001)
    xb = synth.bf16_bits_to_f32(_x(T, K, 83))
    xb[0, K // 2 + 1] = np.inf
    if T > 1:
        xb[T - 1, K - 1] = -np.inf
    if T > 2:  # two in one group
        xb[1] = 0
        xb[1, K - 2], xb[1, K - 7] = 3e37, 2.9e37
    if T > 3:
        xb[2, 0], xb[2, 40] = np.inf, -np.inf
    x = synth.bf16_bits(xb)
    xf = synth.bf16_bits_to_f32(x).astype(np.float64)
    y = torch.empty((T, N), device=dev())
    moe.moe_w4_linear(moe.MOE_INT4, _pack(moe.MOE_INT4, codes, scales, zeros, K, group), N, K, group, to_dev(x), None, y)
    got = y.double().cpu().numpy()
    w, mag = _dequant(moe.MOE_INT4, codes, scales, zeros, K, group)
    with np.errstate(invalid="ignore"):
        for t in range(T):
            far = ~np.isfinite(xf[t])
            ref = np.where(far, 0.0, xf[t]) @ w.T
            if far.any():
                ref = ref + (w[:, far] * xf[t, far]).sum(1)
            else:
                lim = 2 * (2 * K + 64) * U * (mag @ np.abs(xf[t])) + 1e-37
                assert np.isfinite(got[t]).all() and np.all(np.abs(got[t] - ref) <= lim), t
            if far.any():
                np.testing.assert_array_equal(got[t], ref, err_msg=str(t))


def test_the_most_rows():
    """2^30 rows: 2^32 fragments of codes and as many words of scales, one more than a launch can
    have threads.  100 GiB in all; each output has 32 products, so the bound is tight."""
    N, K, group = 1 << 30, 32, 32
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GiB of free device memory")
    g = torch.Generator(device=dev()).manual_seed(9)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=dev(), generator=g)
    scales = torch.full((N, 1), 0.01, dtype=torch.float16, device=dev())
    scales.view(torch.int16).add_(torch.arange(N, device=dev(), dtype=torch.int32).remainder_(257).to(torch.int16)[:, None])
    w = torch.empty(moe.moe_w4_bytes(moe.MOE_INT4, N, K, group), dtype=torch.uint8, device=dev())
    moe.moe_w4_pack(moe.MOE_INT4, codes, scales, None, N, K, group, w)
    x = _x(1, K, 4)
    y = torch.empty((1, N), dtype=torch.bfloat16, device=dev())
    moe.moe_w4_linear(moe.MOE_INT4, w, N, K, group, to_dev(x), None, y)
    torch.cuda.synchronize()
    edge = [b + d for b in (1 << 22, 1 << 28, 1 << 29, 3 << 28) for d in (-17, -1, 0, 16)]
    rows = torch.tensor([0, 1, 15, 16, N - 17, N - 16, N - 1] + edge, device=dev())
    rows = torch.cat([rows, torch.randint(0, N, (4000,), device=dev(), generator=g)])
    wr, mag = _dequant(moe.MOE_INT4, codes[rows].cpu().numpy(), scales[rows].cpu().numpy(), None, K, group)
    _check(y[:, rows], wr, mag, x, None, True, "2^30 rows")
    del codes, scales, w, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,N", [(2, 77), (6, 77), (13, 77), (40, 9003)])
def test_infinite_activations_with_bias_strides_and_bf16(T, N):
    """An output formed again takes its bias and its place in a wider tensor; a bias of -inf (a masked
    row) makes that row -inf for finite tokens; other tokens are those of a batch without the infinite one."""
    K, group = 544, 64
    codes, scales, zeros = _weights(moe.MOE_INT4, N, K, group, seed=91)
    scales[scales == 0] = np.float16(0.001)
    w = _pack(moe.MOE_INT4, codes, scales, zeros, K, group)
    bias = np.random.default_rng(92).standard_normal(N).astype(np.float32)
    bias[5] = -np.inf
    x = to_dev(_x(T, K, 93)).view(torch.bfloat16)
    out = torch.full((T + 1, N + 5), 7.0, dtype=torch.bfloat16, device=dev())
    clean, y = torch.empty((T, N), dtype=torch.bfloat16, device=dev()), out[:T, :N]
    moe.moe_w4_linear(moe.MOE_INT4, w, N, K, group, x, to_dev(bias), clean)
    x[1, 100] = -float("inf")
    moe.moe_w4_linear(moe.MOE_INT4, w, N, K, group, x, to_dev(bias), y)
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(y[keep], clean[keep]) and bool((clean[:, 5] == -float("inf")).all())
    d = _dequant(moe.MOE_INT4, codes, scales, zeros, K, group)[0][:, 100]
    with np.errstate(invalid="ignore"):
        np.testing.assert_array_equal(y[1].float().cpu().numpy(), d * -np.inf + bias)
    assert bool((out[T] == 7).all()) and bool((out[:, N:] == 7).all())
