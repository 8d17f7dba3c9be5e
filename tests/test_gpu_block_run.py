"""The operators around the experts together, as a model runs them: a block of the serving path, and the
forward and backward pass of routed experts whose products are the caller's."""
import pytest
import torch

import plain_ops as P
import synth
from helpers import pool_from_experts, to_dev
from routed_expert_ffn_layer_amd import layer as L
from routed_expert_ffn_layer_amd import moe

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
R, LN = moe.MOE_NORM_RMS, moe.MOE_NORM_LAYER


@pytest.mark.parametrize("wdt,T,shared", [(synth.BF16, 1, 32), (synth.BF16, 9, 0), (synth.BF16, 70, 64), (synth.MXFP4, 3, 0),
                                          (synth.MXFP4, 200, 0), (synth.F32, 5, 0)])
def test_serving_block(wdt, T, shared):
    """Projection back to the hidden size with the residual added in place, then the layer as a block with the next
    block's norm: every step against its plain form on the step's own inputs, the layer against the separate calls."""
    H, I, E, k = 128, 64, 16, 4
    lay = synth.small_layer(wdt, T, H, I, E, k, 77, shared=bool(shared), I_shared=shared)
    dt = F32 if wdt == synth.F32 else BF16
    g = torch.Generator().manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    ctx, w_o, res = n(T, 96).to(dt), (n(H, 96) * 0.1).to(dt), n(T, H)
    w_router, pre_w, post_w, post_b, next_w, gate = (n(E, H) * 0.1).to(dt), 1 + 0.1 * n(H), 1 + 0.1 * n(H), 0.1 * n(H), 1 + 0.1 * n(H), n(H)
    pre, post, nxt = (R, pre_w.cuda()), (LN, post_w.cuda(), post_b.cuda()), (R, next_w.cuda())
    pool, stride = pool_from_experts(lay["experts"])
    sh = to_dev(lay["shared"]) if shared else None
    slots = L.identity_slots(E)
    b = L.BlockBuffers(T, E, k, H, I, wdt, I_shared=shared)
    stream = res.cuda()
    moe.moe_linear(w_o.cuda(), ctx.cuda(), None, moe.MOE_ACT_NONE, stream, stream)
    torch.cuda.synchronize()
    ref, tol = P.linear(ctx, w_o, None, "none", res)
    P.check(stream, ref, P.stored(ref, tol, F32), "projection")
    before = stream.cpu().clone()
    x = L.forward_block(b, stream, w_router.cuda(), pre, post, pool, stride, slots, sh, gate.cuda(), 0.5, 0.9, nxt, 1e-6)
    torch.cuda.synchronize()
    (ref, tol) = P.block_norm(None, None, None, 1.0, before, 1.0, (R, pre_w, None), 1e-6)[1]
    P.check(b.x, ref, P.stored(ref, tol, dt), "layer's input")
    ref, tol = P.linear(b.x.cpu(), w_router, None, "none", None)
    P.check(b.logits, ref, P.stored(ref, tol, F32), "logits")
    c = L.LayerBuffers(T, E, k, H, I, wdt, I_shared=shared)
    (L.forward_decode if L.few_tokens(c) else L.forward)(c, b.logits, b.x, pool, stride, slots, sh)
    torch.cuda.synchronize()
    assert torch.equal(c.y, b.y) and torch.equal(c.topk_ids, b.topk_ids)
    new, out = P.block_norm(b.y.cpu(), (LN, post_w, post_b), gate, 0.5, before, 0.9, (R, next_w, None), 1e-6)
    P.check(stream, new[0], P.stored(*new, F32), "residual stream")
    P.check(x, out[0], P.stored(*out, dt), "next input")
    # a second block from the input that the first one left, without a norm of its own behind it
    kept, inp = stream.cpu().clone(), x.clone()
    back = L.forward_block(b, stream, w_router.cuda(), None, None, pool, stride, slots, sh, x=x)
    torch.cuda.synchronize()
    assert back is stream
    new, _ = P.block_norm(b.y.cpu(), None, None, 1.0, kept, 1.0, None, 1e-6)
    P.check(stream, new[0], P.stored(*new, F32), "second block")
    assert torch.equal(x, inp)


def test_block_captured_and_replayed():
    T, H, I, E, k = 4, 64, 32, 8, 2
    lay = synth.small_layer(synth.BF16, T, H, I, E, k, 5)
    pool, stride = pool_from_experts(lay["experts"])
    g = torch.Generator().manual_seed(0)
    w_router, w = torch.randn(E, H, generator=g).to(BF16).cuda(), torch.ones(H, device="cuda")
    start = torch.randn(T, H, generator=g).to(BF16).cuda()
    slots = L.identity_slots(E)
    one, two = L.BlockBuffers(T, E, k, H, I, synth.BF16), L.BlockBuffers(T, E, k, H, I, synth.BF16)
    run = lambda b, r, st=None: L.forward_block(b, r, w_router, (R, w), (R, w), pool, stride, slots, next_pre=(R, w), stream=st)  # noqa: E731
    a, c = start.clone(), start.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        run(one, a)
    for _ in range(3):
        graph.replay()
        x = run(two, c)
        torch.cuda.synchronize()
        assert torch.equal(a, c) and torch.equal(one.x_next, x)


def test_training_pass():
    """Route, dispatch, the caller's experts (one product each, through moe_linear where an expert has rows), combine,
    and the whole gradient, in f32 against the definition's own in 64 bits.

    Bound: f32 sums over H (twice) and k with a few roundings on the way are off by at most (2 H + k + 16) u of the
    same chain in absolute values; 4 times that for the differences of the softmax's gradient."""
    T, H, E, k = 150, 40, 6, 2
    g = torch.Generator().manual_seed(3)
    x, w_r, dy = torch.randn(T, H, generator=g), torch.randn(E, H, generator=g) * 0.3, torch.randn(T, H, generator=g)
    we = torch.randn(E, H, H, generator=g) * 0.2
    d = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    xd, wd, dyd, wrd = x.cuda(), we.cuda(), dy.cuda(), w_r.cuda()
    logits, ids, w = d(T, E), i(T, k), d(T, k)
    moe.moe_linear(wrd, xd, None, moe.MOE_ACT_NONE, None, logits)
    moe.moe_route_topk(logits, k, ids, w)
    ids[:, 1][torch.arange(T, device="cuda") % 7 == 0] = -1  # pairs past some limit go to no expert
    counts, offsets, order, inv, rows = i(E), i(E + 1), i(T * k), i(T * k), d(T * k, H)
    ws = torch.empty(max(moe.moe_dispatch_workspace(T, k, E), 16), dtype=torch.uint8, device="cuda")
    moe.moe_dispatch(xd, ids, E, counts, offsets, order, inv, rows, ws)
    out, at = d(T * k, H), offsets.tolist()
    for e in range(E):
        moe.moe_linear(wd[e], rows[at[e]:at[e + 1]], None, moe.MOE_ACT_NONE, None, out[at[e]:at[e + 1]])
    y = d(T, H)
    moe.moe_combine_rows(out, w, inv, y)
    d_out, d_w, d_in, d_we = d(T * k, H), d(T, k), d(T * k, H), d(E, H, H)
    moe.moe_combine_rows_backward(dyd, out, w, inv, d_out, d_w)
    for e in range(E):
        part = slice(at[e], at[e + 1])
        moe.moe_linear(wd[e].t().contiguous(), d_out[part], None, moe.MOE_ACT_NONE, None, d_in[part])
        d_we[e] = d_out[part].t() @ rows[part]
    dx, d_logits = d(T, H), d(T, E)
    moe.moe_dispatch_backward(d_in, inv, k, dx)
    moe.moe_gate_backward(ids, w, d_w, d_logits)
    torch.cuda.synchronize()

    idc, live = ids.cpu().long(), ids.cpu() >= 0
    def chain(x, we, dy, wt, sign):
        """y, dx, d_we, d_w of given gate weights; sign -1: differences, +1: everything added up."""
        xe = torch.einsum("th,tkoh->tko", x, we[idc.clamp(min=0)]) * live[..., None]
        yy = (wt[..., None] * xe).sum(1)
        do = wt[..., None] * dy[:, None, :] * live[..., None]
        dwt = (xe * dy[:, None, :]).sum(2)
        dxx = torch.einsum("tko,tkoh->th", do, we[idc.clamp(min=0)])
        dwe = torch.zeros(E, H, H, dtype=torch.float64)
        for e in range(E):
            dwe[e] = torch.einsum("tko,th->oh", do * (idc == e)[..., None], x)
        mean = (wt * dwt).sum(1, keepdim=True)
        return yy, dxx, dwe, dwt, wt * (dwt + sign * mean)

    full = torch.softmax(logits.cpu().double().gather(1, logits.cpu().double().topk(k, 1).indices), 1)
    P.check(w, full, 16 * P.U, "gate weights")
    wt = w.cpu().double()
    ref = chain(x.double(), we.double(), dy.double(), wt, -1)
    mag = chain(x.double().abs(), we.double().abs(), dy.double().abs(), wt, 1)
    u = (2 * H + k + 16) * P.U
    for got, r, m, name in zip((y, dx, d_we, d_w), ref, mag, ("y", "dx", "d_we", "d_w")):
        P.check(got, r, (T * 2 if name == "d_we" else 1) * u * m, name)  # d_we: a library sum over the tokens
    dl, ml = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    t, j = torch.nonzero(live, as_tuple=True)
    dl[t, idc[t, j]], ml[t, idc[t, j]] = ref[4][t, j], mag[4][t, j]
    P.check(d_logits, dl, 4 * u * ml, "d_logits")
