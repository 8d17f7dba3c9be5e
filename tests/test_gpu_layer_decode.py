"""The one-call layer for a few tokens (moe_layer_decode) against the layer computed in
64 bits from the decoded weights.

The bound is element by element, from the roundings the kernels make.  With u = 2^-24 and
exact products of bf16 operands, a K-term sum in f32 in any order is off by at most
2 (K + 64) u times the sum of magnitudes (64 covers the joins; the factor 2 that a matrix
instruction's internal sum need not round to nearest).  So, with |W||x| the sums of
magnitudes,
    dg <= 2 (H + 64) u |Wg||x|,  du <= 2 (H + 64) u |Wu||x|
    dh <= 1.1 dg |up| + |silu| du + |h| (2^-8 or 2^-16 + (8 + |g|) 2^-23)
(|silu'| <= 1.1; the intermediate is rounded to bf16, half a step 2^-8 relative, or up to 8
tokens to two bf16, 2^-16; the hardware exponential and reciprocal), and through the down product and the weights
    dy <= sum_j w_j ( |W2| dh + 2 (I + 64) u |W2||h| ) + (2^-18 + (k + 2) u) sum_j w_j |row_j|
(gate weights good to 2e-6 < 2^-18).  Second order terms are covered by a factor 1.02; a
bf16 output adds 2^-8 |y| (1.02 of it as well).
"""
import numpy as np
import pytest
import torch

import synth
from helpers import W_ATOL, W_RTOL, bf16_to_f64, dev, log, pool_from_experts, to_dev
from routed_expert_ffn_layer_amd import layer as L
from routed_expert_ffn_layer_amd import moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _silu(z):
    return z / (1.0 + np.exp(-z))


def _expert_rows(ora, dtype, slot, H, I, x, half_step):
    """Rows FFN(x) [n][H] and their error bound."""
    wg, wu, wd = ora.decode_expert(dtype, slot, H, I)
    g, u = x @ wg.T, x @ wu.T
    dg, du = (2 * (H + 64) * U * (np.abs(x) @ np.abs(w).T) for w in (wg, wu))
    h = _silu(g) * u
    dh = 1.1 * dg * np.abs(u) + np.abs(_silu(g)) * du + np.abs(h) * (half_step + (8 + np.abs(g)) * 2.0 ** -23)
    return h @ wd.T, (dh + 2 * (I + 64) * U * np.abs(h)) @ np.abs(wd).T


def _reference(ora, lay, ids, w, have=None):
    """y [T][H] and its bound for the routing ids, w (pairs outside `have` left out)."""
    dtype, T, H, I, E, k = (lay[n] for n in ("dtype", "T", "H", "I", "E", "k"))
    half_step = 2.0 ** -16 if T <= 8 else 2.0 ** -8
    x = ora.decode_x(dtype, lay["x"], T, H)
    y, b = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(ids):
        if e < 0 or e >= E or (have is not None and not have[e]):
            continue
        for t, j in zip(*np.nonzero(ids == e)):
            row, d = _expert_rows(ora, dtype, lay["experts"][e], H, I, x[t:t + 1], half_step)
            y[t] += w[t, j] * row[0]
            b[t] += np.abs(w[t, j]) * (d[0] + (2.0 ** -18 + (k + 2) * U) * np.abs(row[0]))
    if lay["shared"] is not None:
        row, d = _expert_rows(ora, dtype, lay["shared"], H, lay["I_shared"], x, half_step)
        y += row
        b += d + (k + 2) * U * np.abs(row)
    return y, 1.02 * b


def _check(y, ref, bound, bf16, what):
    got = bf16_to_f64(y) if bf16 else y.cpu().numpy().astype(np.float64)
    lim = bound + (1.02 * 2.0 ** -8 * np.abs(ref) if bf16 else 0) + 1e-30
    worst = float(np.max(np.abs(got - ref) / lim)) if ref.size else 0.0
    log(f"{what}: error / bound = {worst:.3f}")
    assert worst <= 1.0, what


def _buffers(lay, ydt):
    b = L.LayerBuffers(lay["T"], lay["E"], lay["k"], lay["H"], lay["I"], lay["dtype"], I_shared=lay["I_shared"])
    b.ydt = ydt
    b.y = torch.empty((lay["T"], lay["H"]), dtype=torch.float32 if ydt == moe.MOE_F32 else torch.bfloat16, device=dev())
    return b


def _put(lay):
    pool, stride = pool_from_experts(lay["experts"])
    return (pool, stride, to_dev(lay["shared"]) if lay["shared"] is not None else None, to_dev(lay["x"]),
            to_dev(lay["logits"]))


CASES = [
    # dtype, T, H, I, E, k, I_shared (0: none), logits
    (synth.BF16, 1, 256, 128, 16, 4, 128, "normal"),
    (synth.BF16, 1, 32, 32, 1, 1, 0, "normal"),       # the smallest shape
    (synth.BF16, 2, 96, 160, 5, 5, 32, "normal"),     # every expert active, ragged tiles
    (synth.BF16, 16, 288, 96, 37, 7, 224, "normal"),  # a shared expert wider than the routed ones
    (synth.BF16, 17, 64, 64, 300, 8, 64, "zipf"),     # shared tokens in two runs
    (synth.BF16, 64, 128, 32, 8, 8, 0, "normal"),     # every expert has all 64 tokens: four runs each
    (synth.BF16, 16, 64, 32, 64, 32, 32, "normal"),   # 512 pairs, k = 32
    (synth.BF16, 3, 2048, 512, 12, 8, 512, "normal"),
    (synth.MXFP4, 1, 256, 128, 16, 6, 0, "normal"),
    (synth.MXFP4, 1, 32, 32, 2, 2, 32, "normal"),     # less than one column step
    (synth.MXFP4, 5, 160, 96, 9, 3, 0, "normal"),     # columns past the last whole step
    (synth.MXFP4, 8, 2176, 288, 24, 6, 64, "zipf"),   # a second scale block
    (synth.MXFP4, 33, 128, 416, 40, 6, 0, "zipf"),
    (synth.MXFP4, 64, 256, 64, 1024, 8, 0, "zipf"),   # 512 pairs, the most experts
    (synth.MXFP4, 64, 96, 32, 1, 1, 0, "normal"),     # one expert for all
    (synth.MXFP4, 4, 4096, 2048, 8, 2, 0, "normal"),
    (synth.MXFP4, 40, 4096, 96, 6, 3, 32, "normal"),  # fewer token rows in LDS than a matrix tile holds
    (synth.BF16, 21, 8192, 64, 3, 2, 32, "normal"),   # fewer still: runs of 7
    (synth.BF16, 3, 65536, 32, 2, 1, 0, "normal"),    # one row at a time
]


@pytest.mark.parametrize("ydt", [moe.MOE_F32, moe.MOE_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(str(v) for v in c))
def test_layer_against_64_bits(ora, case, ydt):
    dtype, T, H, I, E, k, ish, logits = case
    log(f"layer_decode {case} ydt={ydt}")
    lay = synth.small_layer(dtype, T, H, I, E, k, seed=T + H + E, shared=ish > 0, I_shared=ish, logits=logits)
    pool, stride, sh, x, lg = _put(lay)
    b = _buffers(lay, ydt)
    L.forward_decode(b, lg, x, pool, stride, L.identity_slots(E), sh)
    torch.cuda.synchronize()
    ids, _, w64 = ora.route_topk(lay["logits"], k)
    np.testing.assert_array_equal(b.topk_ids.cpu().numpy(), ids)
    np.testing.assert_allclose(b.topk_w.cpu().numpy(), w64, rtol=W_RTOL, atol=W_ATOL)
    ref, bound = _reference(ora, lay, ids, w64)
    _check(b.y, ref, bound, ydt == moe.MOE_BF16, str(case))


@pytest.mark.parametrize("dtype", [synth.BF16, synth.MXFP4])
def test_ties_and_tied_extremes(ora, dtype):
    T, H, I, E, k = 6, 64, 32, 130, 8
    lay = synth.small_layer(dtype, T, H, I, E, k, seed=5)
    lg = lay["logits"]
    lg[0] = 0.0
    lg[1] = -0.0
    lg[1, ::2] = 0.0
    lg[2] = np.finfo(np.float32).min
    lg[3, 100:] = np.finfo(np.float32).max
    lg[4, ::3] = lg[4, 0]
    pool, stride, sh, x, lgd = _put(lay)
    b = _buffers(lay, moe.MOE_F32)
    L.forward_decode(b, lgd, x, pool, stride, L.identity_slots(E), sh)
    torch.cuda.synchronize()
    ids, _, w64 = ora.route_topk(lg, k)
    np.testing.assert_array_equal(b.topk_ids.cpu().numpy(), ids)
    ref, bound = _reference(ora, lay, ids, w64)
    _check(b.y, ref, bound, False, "ties")


@pytest.mark.parametrize("dtype", [synth.BF16, synth.MXFP4])
@pytest.mark.parametrize("shared", [False, True])
def test_experts_without_a_slot_contribute_nothing(ora, dtype, shared):
    T, H, I, E, k = 9, 96, 64, 12, 4
    lay = synth.small_layer(dtype, T, H, I, E, k, seed=31, shared=shared, I_shared=32)
    pool, stride, sh, x, lg = _put(lay)
    ids, _, w64 = ora.route_topk(lay["logits"], k)
    # half the experts, in slots of another order; then none at all
    perm = torch.randperm(E, generator=torch.Generator().manual_seed(1))
    mixed = torch.empty_like(pool)
    mixed[perm.to(dev())] = pool
    slots = perm.to(torch.int32)
    slots[::2] = -1
    for table, have in ((slots, (slots >= 0).numpy()), (torch.full((E,), -1, dtype=torch.int32), np.zeros(E, bool))):
        b = _buffers(lay, moe.MOE_F32)
        b.workspace.fill_(255)  # NaN intermediates: none may be read
        L.forward_decode(b, lg, x, mixed, stride, table.to(dev()), sh)
        torch.cuda.synchronize()
        ref, bound = _reference(ora, lay, ids, w64, have)
        _check(b.y, ref, bound, False, f"{int(have.sum())} of {E} experts")
        if not shared and not have.any():
            assert torch.equal(b.y, torch.zeros_like(b.y))


@pytest.mark.parametrize("dtype", [synth.BF16, synth.MXFP4])
def test_given_routing(ora, dtype):
    """The caller's ids and weights: an expert twice in one token, ids outside the
    experts, weights that do not sum to one, one of them zero."""
    T, H, I, E, k = 20, 128, 96, 6, 5
    lay = synth.small_layer(dtype, T, H, I, E, k, seed=77, shared=True, I_shared=64)
    pool, stride, sh, x, _ = _put(lay)
    g = np.random.default_rng(3)
    ids = g.integers(0, E, (T, k)).astype(np.int32)
    ids[0] = 2          # the same expert in every place
    ids[1, 1] = ids[1, 0]
    ids[2] = [-1, E, 1, 2 ** 30, -2 ** 31]
    ids[3] = -7
    w = g.standard_normal((T, k)).astype(np.float32)
    w[4, 2] = 0.0
    b = _buffers(lay, moe.MOE_F32)
    b.topk_ids.copy_(torch.from_numpy(ids))
    b.topk_w.copy_(torch.from_numpy(w))
    L.forward_decode(b, None, x, pool, stride, L.identity_slots(E), sh)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(b.topk_ids.cpu().numpy(), ids)
    np.testing.assert_array_equal(b.topk_w.cpu().numpy(), w)
    ref, bound = _reference(ora, lay, ids, w.astype(np.float64))
    _check(b.y, ref, bound, False, "given routing")


def test_given_routing_of_moe_route_equals_own_routing():
    """moe_route's ids are the layer's own, and its gate weights differ by the order of one
    sum: k positive terms, the same on both sides, added with k - 1 roundings each and
    divided with one, so by at most 2 k u relative (second order below the last u counted,
    as the largest term is exactly 1 and enters without rounding).  The layer on given
    routing equals the layer that made it, bit for bit."""
    k = 4
    lay = synth.small_layer(synth.BF16, 8, 128, 64, 32, k, seed=8, shared=True, I_shared=64)
    pool, stride, sh, x, lg = _put(lay)
    b, c = _buffers(lay, moe.MOE_BF16), _buffers(lay, moe.MOE_BF16)
    L.forward_decode(b, lg, x, pool, stride, L.identity_slots(32), sh)
    L.route(c, lg)
    torch.cuda.synchronize()
    assert torch.equal(b.topk_ids, c.topk_ids)
    assert bool(((b.topk_w - c.topk_w).abs() <= 2 * k * U * c.topk_w).all())
    c.topk_w.copy_(b.topk_w)
    L.forward_decode(c, None, x, pool, stride, L.identity_slots(32), sh)
    torch.cuda.synchronize()
    assert torch.equal(b.y.view(torch.int16), c.y.view(torch.int16))


def test_rows_behind_the_batch_stay():
    lay = synth.small_layer(synth.MXFP4, 3, 96, 64, 8, 2, seed=9)
    pool, stride, sh, x, lg = _put(lay)
    b = _buffers(lay, moe.MOE_BF16)
    big = [torch.full((s[0] + 2, s[1]), 7, dtype=d, device=dev())
           for s, d in (((3, 96), torch.bfloat16), ((3, 2), torch.int32), ((3, 2), torch.float32))]
    need = moe.moe_layer_decode_workspace(3, 2, 8, 96, 64, 0, b.wdt)
    ws = torch.full((need + 64,), 7, dtype=torch.uint8, device=dev())
    moe.moe_layer_decode(b.wdt, pool, stride, L.identity_slots(8), None, 0, x, lg, 3, 2, 8, 96, 64, big[1], big[2],
                         big[0], moe.MOE_BF16, ws)
    torch.cuda.synchronize()
    for t in big:
        assert bool((t[3:] == 7).all()) and not bool((t[:3] == 7).all())
    assert bool((ws[need:] == 7).all())


def test_a_bad_token_stays_its_own():
    """NaN and infinity in one token's activations reach that token's row only."""
    lay = synth.small_layer(synth.MXFP4, 6, 160, 64, 4, 4, seed=10)
    pool, stride, sh, x, lg = _put(lay)
    b = _buffers(lay, moe.MOE_F32)
    clean = L.forward_decode(b, lg, x, pool, stride, L.identity_slots(4), sh).clone()
    x = x.view(torch.bfloat16).clone()
    x[2, 5], x[4, 100] = float("nan"), float("inf")
    y = L.forward_decode(b, lg, x, pool, stride, L.identity_slots(4), sh)
    torch.cuda.synchronize()
    for t in (0, 1, 3, 5):
        assert torch.equal(y[t], clean[t])
    assert bool(torch.isnan(y[2]).all())


def test_slots_past_4_gib(ora):
    lay = synth.small_layer(synth.BF16, 2, 64, 32, 3, 3, seed=12)
    stride = (3 << 30) + 256
    pool = torch.empty(2 * stride + lay["experts"].shape[1], dtype=torch.uint8, device=dev())
    for e in range(3):
        pool[e * stride:e * stride + lay["experts"].shape[1]] = to_dev(lay["experts"][e])
    b = _buffers(lay, moe.MOE_F32)
    L.forward_decode(b, to_dev(lay["logits"]), to_dev(lay["x"]), pool, stride, L.identity_slots(3))
    torch.cuda.synchronize()
    ids, _, w64 = ora.route_topk(lay["logits"], 3)
    ref, bound = _reference(ora, lay, ids, w64)
    _check(b.y, ref, bound, False, "slots past 4 GiB")


@pytest.mark.parametrize("dtype,T,shared", [(synth.BF16, 4, True), (synth.MXFP4, 1, False), (synth.MXFP4, 40, True)])
def test_replays_streams_and_two_calls_at_once(dtype, T, shared):
    """A captured call replayed with new inputs, eager work between the replays; a call on
    another stream; two calls running side by side, each with buffers of its own: all
    equal the eager call bit for bit."""
    H, I, E, k, ish = 512, 256, 16, 4, 64 if shared else 0
    lays = [synth.small_layer(dtype, T, H, I, E, k, seed=900 + i, shared=shared, I_shared=ish) for i in range(3)]
    pool, stride, sh, _, _ = _put(lays[0])
    slots = L.identity_slots(E)
    xs, lgs = [to_dev(a["x"]) for a in lays], [to_dev(a["logits"]) for a in lays]
    refs = []
    for x, lg in zip(xs, lgs):
        refs.append(L.forward_decode(_buffers(lays[0], moe.MOE_BF16), lg, x, pool, stride, slots, sh).view(torch.int16))
    torch.cuda.synchronize()
    x_s, lg_s, bg = xs[0].clone(), lgs[0].clone(), _buffers(lays[0], moe.MOE_BF16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward_decode(bg, lg_s, x_s, pool, stride, slots, sh)
    for rep in range(4):
        i = (rep + 1) % 3
        x_s.copy_(xs[i])
        lg_s.copy_(lgs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bg.y.view(torch.int16), refs[i]), rep
        j = (i + 1) % 3
        again = L.forward_decode(_buffers(lays[0], moe.MOE_BF16), lgs[j], xs[j], pool, stride, slots, sh)
        assert torch.equal(again.view(torch.int16), refs[j])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    b1, b2 = _buffers(lays[0], moe.MOE_BF16), _buffers(lays[0], moe.MOE_BF16)
    for _ in range(5):
        L.forward_decode(b1, lgs[1], xs[1], pool, stride, slots, sh, stream=s1)
        L.forward_decode(b2, lgs[2], xs[2], pool, stride, slots, sh, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(b1.y.view(torch.int16), refs[1]) and torch.equal(b2.y.view(torch.int16), refs[2])


def test_no_tokens():
    b = L.LayerBuffers(0, 8, 2, 64, 32, moe.MOE_BF16)
    z = torch.zeros(64, dtype=torch.uint8, device=dev())
    moe.moe_layer_decode(moe.MOE_BF16, z, 1 << 20, z, None, 0, z, z, 0, 2, 8, 64, 32, z, z, z, moe.MOE_F32, b.workspace)
    torch.cuda.synchronize()


def test_close_to_the_separate_calls():
    """The same layer through route, grouped FFN and combine."""
    lay = synth.small_layer(synth.MXFP4, 12, 512, 256, 32, 6, seed=4, shared=True, I_shared=128)
    pool, stride, sh, x, lg = _put(lay)
    b, c = _buffers(lay, moe.MOE_F32), _buffers(lay, moe.MOE_F32)
    L.forward_decode(b, lg, x, pool, stride, L.identity_slots(32), sh)
    L.forward(c, lg, x, pool, stride, L.identity_slots(32), sh)
    torch.cuda.synchronize()
    assert torch.equal(b.topk_ids, c.topk_ids)
    # an intermediate near a rounding border may round to either side: 2^-8 of it, both ways
    scale = c.y.pow(2).mean().sqrt()
    assert float((b.y - c.y).abs().max()) <= 2 * 2 ** -8 * float(scale) * 4
