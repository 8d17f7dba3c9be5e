"""The parts that the few-token operators cut their sums into: every part of K of the layer's two
products, every wave's share of a long 4-bit product, and codes past 4 GiB.

A bound that grows with K says little where K is long: a part could be missing and the result still
lie within it.  So the layer's cases are chosen narrow enough, and each is checked to be: with any one
column step of the tokens, or of the intermediate, left out of the reference, it would miss its own
bound.  The products take integers, whose sums are exact in f32 in any order (below 2^24 of their
unit), and are compared for equality.
"""
import numpy as np
import pytest
import torch

import synth
from helpers import dev, log, to_dev
from routed_expert_ffn_layer_amd import layer as L
from routed_expert_ffn_layer_amd import moe
from test_gpu_layer_decode import U, _buffers, _check, _put, _reference, _silu

pytestmark = pytest.mark.gpu


def _every_step_matters(ora, lay, ids, w, lim):
    """Leaves each column step out of W13's sums (all tokens' x), then out of W2's, and requires
    that some output moves by more than its bound."""
    dtype, T, H, I, E = (lay[n] for n in ("dtype", "T", "H", "I", "E"))
    x = ora.decode_x(dtype, lay["x"], T, H)
    ks = 128 if dtype == synth.MXFP4 else 32
    users = []  # (weights of the matrices, rows of x, their factors)
    for e in np.unique(ids):
        if 0 <= e < E:
            f = np.where(ids == e, w, 0.0).sum(1)
            t = np.nonzero((ids == e).any(1))[0]
            users.append((ora.decode_expert(dtype, lay["experts"][e], H, I), t, f[t]))
    if lay["shared"] is not None:
        users.append((ora.decode_expert(dtype, lay["shared"], H, lay["I_shared"]), np.arange(T), np.ones(T)))
    worst = np.inf
    widest = max(I, lay["I_shared"])
    for matrix, width in (("W13", H), ("W2", widest)):
        for k0 in range(0, width, ks):
            if matrix == "W13" and not x[:, k0:k0 + ks].any():
                continue
            moved = np.zeros((T, H))
            for (wg, wu, wd), t, f in users:
                g, u = x[t] @ wg.T, x[t] @ wu.T
                h = _silu(g) * u
                if matrix == "W13":
                    part = x[t][:, k0:k0 + ks]
                    h = h - _silu(g - part @ wg[:, k0:k0 + ks].T) * (u - part @ wu[:, k0:k0 + ks].T)
                    moved[t] += f[:, None] * (h @ wd.T)
                else:
                    moved[t] += f[:, None] * (h[:, k0:k0 + ks] @ wd[:, k0:k0 + ks].T)
            worst = min(worst, float(np.max(np.abs(moved) / lim)))
    log(f"least step moves an output by {worst:.2f} bounds")
    assert worst > 1.0


CASES = [
    # dtype, T, H, I, E, k, I_shared
    # W2 in parts: half tiles (H <= 2048), h in two parts of bf16 (T <= 8), then in one
    (synth.MXFP4, 1, 256, 1056, 4, 2, 0),     # 9 column steps: an odd number, the last one alone
    (synth.MXFP4, 4, 256, 1056, 4, 2, 0),
    (synth.MXFP4, 8, 256, 1056, 4, 1, 416),   # a shared expert of 4 steps in the same parts
    (synth.MXFP4, 9, 256, 1056, 4, 1, 0),
    (synth.MXFP4, 12, 96, 2080, 4, 2, 0),
    (synth.MXFP4, 2, 64, 4128, 2, 1, 0),      # 33 steps, a third scale block
    (synth.BF16, 1, 256, 1056, 4, 2, 0),      # 33 steps of 32
    (synth.BF16, 8, 160, 544, 4, 2, 96),
    (synth.BF16, 12, 256, 1056, 4, 2, 0),
    # whole tiles (H > 2048)
    (synth.MXFP4, 1, 2080, 1056, 4, 2, 0),
    (synth.MXFP4, 8, 2080, 800, 4, 1, 0),
    (synth.MXFP4, 9, 2080, 1056, 4, 1, 0),
    (synth.MXFP4, 24, 2080, 544, 5, 3, 0),    # one part, several chunks of steps
    (synth.BF16, 1, 2080, 288, 4, 4, 0),
    (synth.BF16, 2, 2080, 544, 4, 2, 0),
    (synth.BF16, 4, 2080, 288, 4, 2, 160),
    (synth.BF16, 9, 2080, 544, 4, 2, 0),
    (synth.BF16, 33, 2080, 160, 5, 4, 0),
]


def _layer(case):
    dtype, T, H, I, E, k, ish = case
    lay = synth.small_layer(dtype, T, H, I, E, k, seed=300 + T + H + I, shared=ish > 0, I_shared=ish)
    if H > 2048:  # the bound of W13's sums goes with H: few columns other than zero keep it small
        lay["x"][:, np.arange(H) % 8 != 5] = 0
    return lay


@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(str(v) for v in c))
def test_parts_of_k(ora, case):
    dtype, T, H, I, E, k, ish = case
    log(f"parts {case}")
    lay = _layer(case)
    ids, _, w64 = ora.route_topk(lay["logits"], k)
    ref, bound = _reference(ora, lay, ids, w64)
    _every_step_matters(ora, lay, ids, w64, bound)
    pool, stride, sh, x, lg = _put(lay)
    b = _buffers(lay, moe.MOE_F32)
    L.forward_decode(b, lg, x, pool, stride, L.identity_slots(E), sh)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(b.topk_ids.cpu().numpy(), ids)
    _check(b.y, ref, bound, False, str(case))


@pytest.mark.parametrize("dtype", [synth.BF16, synth.MXFP4])
def test_the_widest_tokens(ora, dtype):
    """H = 65536 with few columns other than zero (both ends, and one in each quarter and around
    its border), so that the sums of magnitudes stay short."""
    T, H, I, E, k = 3, 65536, 32, 2, 1
    lay = synth.small_layer(dtype, T, H, I, E, k, seed=400)
    keep = [0, 33, 16383, 16384, 20000, 32767, 32768, 40001, 49151, 49152, 60000, 65535]
    x = np.zeros_like(lay["x"])
    x[:, keep] = lay["x"][:, keep]
    lay["x"] = x
    ids, _, w64 = ora.route_topk(lay["logits"], k)
    ref, bound = _reference(ora, lay, ids, w64)
    _every_step_matters(ora, lay, ids, w64, bound)
    pool, stride, sh, xd, lg = _put(lay)
    b = _buffers(lay, moe.MOE_F32)
    L.forward_decode(b, lg, xd, pool, stride, L.identity_slots(E), sh)
    torch.cuda.synchronize()
    _check(b.y, ref, bound, False, f"H = 65536 dtype {dtype}")


@pytest.mark.parametrize("dtype", [synth.BF16, synth.MXFP4])
@pytest.mark.parametrize("T,k,shared", [(1, 6, False), (6, 6, True), (8, 8, False), (12, 5, True), (64, 1, False)])
def test_given_routing_of_few_pairs(ora, dtype, T, k, shared):
    """At most 64 pairs are grouped by one wave: an expert in several places of a token, ids outside the
    experts, tokens with none left, weights that do not sum to one."""
    H, I, E = 96, 160, 9
    lay = synth.small_layer(dtype, T, H, I, E, k, seed=500 + T + k, shared=shared, I_shared=64 if shared else 0)
    g = np.random.default_rng(T + k)
    ids = g.integers(0, E, (T, k)).astype(np.int32)
    ids[0] = 3  # one expert in every place
    w = g.standard_normal((T, k)).astype(np.float32)
    if T > 2:
        ids[1] = -1
        ids[T - 1] = 2 ** 31 - 1
        ids[T // 2, 0] = E
        ids[2, k - 1] = ids[2, 0]
        w[2, 0] = 0.0
    pool, stride, sh, x, _ = _put(lay)
    b = _buffers(lay, moe.MOE_F32)
    b.workspace.fill_(255)  # NaN: nothing of it may be read before it is written
    b.topk_ids.copy_(torch.from_numpy(ids))
    b.topk_w.copy_(torch.from_numpy(w))
    L.forward_decode(b, None, x, pool, stride, L.identity_slots(E), sh)
    torch.cuda.synchronize()
    ref, bound = _reference(ora, lay, ids, w.astype(np.float64))
    _check(b.y, ref, bound, False, f"given routing T={T} k={k}")
    if T > 2 and not shared:
        assert not bool(b.y[1].any()) and not bool(b.y[T - 1].any())
    np.testing.assert_array_equal(b.topk_ids.cpu().numpy(), ids)


FORMATS = [(moe.MOE_MXFP4, 32), (moe.MOE_INT4, 32), (moe.MOE_INT4, 64), (moe.MOE_INT4, 128)]
_E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def _integers(fmt, group, T, N, K, seed):
    """Codes, scales, zeros and x whose sums are whole multiples of 1/4 below 2^22: |x| <= 1, |W| <= 6
    (MXFP4) or 15, also in the two sums (of x q and of x z) that INT4 keeps, and K <= 2^17 = 131072
    gives 15 * 2^17 < 2^21."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    rnd = lambda lo, hi, shape: torch.randint(lo, hi, shape, dtype=torch.uint8, device=dev(), generator=g)
    codes = rnd(0, 256, (N, K // 2))
    n = -(-K // group)
    if fmt == moe.MOE_MXFP4:
        scales, zeros = rnd(126, 128, (N, n)), None  # 1/2 and 1
    else:
        scales, zeros = (rnd(0, 2, (N, n)).half() + 1) / 2, rnd(0, 16, (N, n))
    x = rnd(0, 3, (T, K)).to(torch.bfloat16) - 1
    return codes, scales, zeros, x


def _exact(fmt, group, codes, scales, zeros, x, bias=None):
    """y in 64 bits, some rows of W at a time."""
    N, K = codes.shape[0], x.shape[1]
    y = torch.empty((x.shape[0], N), dtype=torch.float64, device=dev())
    step = max(16, (1 << 28) // K)
    for n in range(0, N, step):
        c = codes[n:n + step]
        q = torch.stack((c & 15, c >> 4), dim=-1).flatten(1)
        per = lambda t: t.double().repeat_interleave(group, 1)[:, :K]
        if fmt == moe.MOE_MXFP4:
            w = _E2M1.to(dev())[q.int()] * per(torch.exp2(scales[n:n + step].double() - 127))
        else:
            w = (q.double() - per(zeros[n:n + step])) * per(scales[n:n + step])
        y[:, n:n + step] = x.double() @ w.t().contiguous()
    return y


def _product(fmt, group, T, N, K, dtype=torch.float32):
    codes, scales, zeros, x = _integers(fmt, group, T, N, K, seed=T + N + K)
    w = torch.empty(moe.moe_w4_bytes(fmt, N, K, group), dtype=torch.uint8, device=dev())
    moe.moe_w4_pack(fmt, codes, scales, zeros, N, K, group, w)
    y = torch.empty((T, N), dtype=dtype, device=dev())
    moe.moe_w4_linear(fmt, w, N, K, group, x, None, y)
    ref = _exact(fmt, group, codes, scales, zeros, x)
    assert float(ref.abs().max()) < 2 ** 22
    return y, ref


@pytest.mark.parametrize("fmt,group", FORMATS, ids=["mxfp4", "int4_32", "int4_64", "int4_128"])
@pytest.mark.parametrize("T,N,K", [(1, 40, 32), (1, 2048, 2048), (4, 1003, 2080), (7, 500, 4096), (16, 100, 4000), (1, 200, 8192),
                                   (8, 300, 6112), (16, 100, 8192), (3, 64, 9024), (6, 40, 12288), (12, 33, 16384),
                                   (2, 48, 131072), (16, 48, 131072), (20, 40, 131072), (24, 6000, 2080), (64, 5000, 4096),
                                   (20, 45003, 416), (64, 33000, 1056), (70, 45000, 288)])
def test_products_of_integers(fmt, group, T, N, K):
    y, ref = _product(fmt, group, T, N, K)
    assert torch.equal(y.double(), ref)


@pytest.mark.parametrize("fmt,group", FORMATS, ids=["mxfp4", "int4_32", "int4_64", "int4_128"])
@pytest.mark.parametrize("T", [5, 40])
def test_products_of_integers_in_bf16(fmt, group, T):
    """The one rounding of an exact sum, to the nearest and ties to even."""
    y, ref = _product(fmt, group, T, 5000, 2080, torch.bfloat16)
    assert torch.equal(y, ref.float().to(torch.bfloat16))


@pytest.mark.parametrize("fmt,group,T", [(moe.MOE_MXFP4, 32, 2), (moe.MOE_INT4, 128, 2), (moe.MOE_INT4, 32, 16),
                                         (moe.MOE_MXFP4, 32, 20), (moe.MOE_INT4, 64, 40)])
def test_every_row_past_4_gib(fmt, group, T):
    """More than 2^32 bytes of codes: every output, not those of a few rows."""
    y, ref = _product(fmt, group, T, 70000, 131072)
    assert torch.equal(y.double(), ref)


@pytest.mark.parametrize("T", [1, 7, 16, 40])
def test_e8m0_scales_at_the_ends(T):
    """E2M1 times 2^(scale - 127) is exact from the smallest scale (a bf16 subnormal of two bits) up, infinite
    from 2^128 on, and NaN for 255; one product an output, so each is exact."""
    N, K = 16, 64
    mags = _E2M1[:8]
    for s in (0, 1, 2, 127, 252, 253, 254, 255):
        codes = torch.zeros((N, K // 2), dtype=torch.uint8, device=dev())
        codes[:8, 0] = torch.arange(8, device=dev()).to(torch.uint8)
        scales = torch.full((N, 2), s, dtype=torch.uint8, device=dev())
        scales[:, 1] = 127
        w = torch.empty(moe.moe_w4_bytes(moe.MOE_MXFP4, N, K, 32), dtype=torch.uint8, device=dev())
        moe.moe_w4_pack(moe.MOE_MXFP4, codes, scales, None, N, K, 32, w)
        x = torch.zeros((T, K), dtype=torch.bfloat16, device=dev())
        x[:, 0] = 2.0 ** -20 if s > 200 else 2.0 ** 20
        y = torch.empty((T, N), device=dev())
        moe.moe_w4_linear(moe.MOE_MXFP4, w, N, K, 32, x, None, y)
        wv = mags * 2.0 ** (s - 127) if s < 255 else torch.full((8,), float("nan"), dtype=torch.float64)
        wv = torch.where(wv >= 2.0 ** 128, float("inf"), wv)
        torch.testing.assert_close(y[:, :8].double().cpu(), (wv * float(x[0, 0])).expand(T, 8), rtol=0, atol=0, equal_nan=True)
