"""The gate's gradient where pairs go to no expert: the softmax holds them all the same, so their logits have one too."""
import pytest
import torch

import plain_ops as P
from routed_expert_ffn_layer_amd import moe

pytestmark = pytest.mark.gpu
T, K, E, H = 60, 3, 12, 24


def _step(x, ids, w, marked, scale, dy):
    """d_topk_w and y of dispatch -> an expert scaling its rows -> combine, the pairs as `marked` has them."""
    i = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offsets, order, inv = i(E), i(E + 1), i(T * K), i(T * K)
    rows, y, d_w = torch.zeros((T * K, H), device="cuda"), torch.zeros((T, H), device="cuda"), torch.zeros((T, K), device="cuda")
    moe.moe_dispatch(x, marked, E, counts, offsets, order, inv, rows)
    n = int(offsets[-1])
    expert = ids.reshape(-1)[order[:n].long()].long()
    rows[:n] *= scale[expert][:, None]
    moe.moe_combine_rows(rows, w, inv, y)
    moe.moe_combine_rows_backward(dy, rows, w, inv, rows, d_w)
    return y, d_w


def _state():
    g = torch.Generator().manual_seed(11)
    x, logits, dy = (torch.randn(*s, generator=g).cuda() for s in ((T, H), (T, E), (T, H)))
    scale = (1 + torch.rand(E, generator=g)).cuda()
    ids, w = torch.zeros((T, K), dtype=torch.int32, device="cuda"), torch.zeros((T, K), device="cuda")
    moe.moe_route_topk(logits, K, ids, w)
    return x, logits, dy, scale, ids, w


def _reference(x, logits, dy, scale, ids, live):
    """Central differences of the loss sum(dy y) by every logit, in 64 bits, and the magnitude that its bound takes."""
    x, logits, dy, scale, ids, live = (t.cpu() for t in (x, logits, dy, scale, ids, live))
    out = scale.double()[ids.long()] * live  # an expert's factor of each pair, 0 for the dropped
    dots = (x.double() * dy.double()).sum(1, keepdim=True) * out  # d loss / d w

    def loss(logits):  # by token: a logit acts on its own token alone
        return (torch.softmax(logits.gather(1, ids.long()), 1) * dots).sum(1)

    h, diff = 1e-5, torch.zeros((T, E), dtype=torch.float64)
    for e in range(E):
        step = torch.zeros(E, dtype=torch.float64)
        step[e] = h
        diff[:, e] = (loss(logits.double() + step) - loss(logits.double() - step)) / (2 * h)
    w = torch.softmax(logits.double().gather(1, ids.long()), 1)
    mag = (x.double() * dy.double()).abs().sum(1, keepdim=True) * out
    # d_w: H + 1 roundings of mag; the weights 16 u; products, sum over k and difference K + 4
    tol = torch.zeros((T, E), dtype=torch.float64)
    tol.scatter_add_(1, ids.long(), w * (mag + (w * mag).sum(1, keepdim=True)) * (2 * H + K + 48) * P.U)
    # differences: h^2 / 6 of a third derivative below 20 |dots|, 2^-52 |loss| / h of rounding
    tol += dots.abs().sum(1, keepdim=True) * (4 * h * h + 2.0 ** -50 / h)
    return diff, tol


def test_limit_on_pairs():
    """Every fifth pair past a limit, every pair of a few tokens: against differences by every logit, the dropped included."""
    x, logits, dy, scale, ids, w = _state()
    marked = ids.clone()
    marked.view(-1)[::5] = -1
    marked[7], marked[20] = -1, E
    live = (marked >= 0) & (marked < E)
    _, d_w = _step(x, ids, w, marked, scale, dy)
    d_logits = torch.empty((T, E), device="cuda")
    moe.moe_gate_backward(ids, w, d_w, d_logits)
    torch.cuda.synchronize()
    diff, tol = _reference(x, logits, dy, scale, ids, live)
    P.check(d_logits, diff, tol)
    # the dropped pairs of tokens that kept one have a gradient; the marked ids lose it
    some = (~live & live.any(1, keepdim=True)).cpu()
    at_dropped = d_logits.cpu().gather(1, ids.cpu().long())[some]
    assert some.sum() > 20 and (at_dropped != 0).all()
    moe.moe_gate_backward(marked, w, d_w, d_logits)
    torch.cuda.synchronize()
    assert not d_logits.cpu().gather(1, ids.cpu().long())[some].any()
    with pytest.raises(AssertionError):
        P.check(d_logits, diff, tol)


def test_shards_add_up():
    """Two shards of the experts, each with the other's pairs marked: their gradients together are the whole."""
    x, logits, dy, scale, ids, w = _state()
    total, part, y = (torch.zeros(s, device="cuda") for s in ((T, E), (T, E), (T, H)))
    for lo, hi in ((0, 5), (5, E)):
        marked = torch.where((ids >= lo) & (ids < hi), ids, torch.full_like(ids, -1))
        one, d_w = _step(x, ids, w, marked, scale, dy)
        moe.moe_gate_backward(ids, w, d_w, part)
        total += part
        y += one
    torch.cuda.synchronize()
    diff, tol = _reference(x, logits, dy, scale, ids, torch.ones_like(ids, dtype=torch.bool))
    P.check(total, diff, 2 * tol)
