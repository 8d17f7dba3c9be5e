"""The sorted tokens' calls where a workgroup holds a token (rows of more than 1024 elements), with more than 8 pairs a token,
rows that end inside a group of 8 at odd strides; and rows so many that they pass the caches by.  Against 64 bits."""
import pytest
import torch

import plain_ops as P
from routed_expert_ffn_layer_amd import moe

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
MARK = 77.0  # what rows hold that no pair goes to


def _wide(v, pad):
    wide = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=v.dtype, device="cuda")
    wide[:, :v.shape[1]] = v
    return wide[:, :v.shape[1]]


def _close(got, ref, tol):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}"


def _pairs(rows, inv, n_rows, T, k):
    """Rows of the pairs in 64 bits, 0 for those without one, [T][k][H]."""
    at = inv.long().view(T, k)
    live = (at >= 0) & (at < n_rows)
    return torch.where(live[..., None], rows.double()[at.clamp(0, n_rows - 1)], 0.0), live


def _all_calls(T, k, E, H, dt, ydt, drop, pad, fewer):
    """The five calls on one order; `fewer` rows less than pairs."""
    g = torch.Generator(device="cuda").manual_seed(T + H)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ids = n(T, E).topk(k, 1).indices.to(torch.int32)
    ids[torch.rand((T, k), generator=g, device="cuda") < drop] = -1
    counts, offsets, order, inv = (t.cuda() for t in P.order(ids.cpu(), E))
    n_rows = T * k - fewer
    # there
    x = _wide(n(T, H).to(dt), pad)
    got = [torch.full_like(t, -7) for t in (counts, offsets, order, inv)]
    rows = _wide(torch.full((n_rows, H), MARK, dtype=dt), pad)
    ws = torch.empty(moe.moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda")
    moe.moe_dispatch(x, ids, E, *got, rows, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (counts, offsets, order, inv)))
    placed = min(int(offsets[-1]), n_rows)
    assert torch.equal(rows[:placed], x[order[:placed].long() // k]) and (rows[placed:] == MARK).all()
    # back
    rows, w = _wide(n(n_rows, H).to(dt), pad), torch.softmax(n(T, k), 1)
    y, dx = (_wide(torch.zeros((T, H), dtype=ydt), pad) for _ in range(2))
    moe.moe_combine_rows(rows, w, inv, y)
    moe.moe_dispatch_backward(rows, inv, k, dx)
    torch.cuda.synchronize()
    mine, live = _pairs(rows, inv, n_rows, T, k)
    for out, v in ((y, w.double()[..., None] * mine), (dx, mine)):
        ref = v.sum(1)
        _close(out, ref, P.stored(ref, k * P.U * v.abs().sum(1), ydt))  # k fused multiply-adds
    # gradients, apart from the rows and in their place
    dy = _wide(n(T, H).to(ydt), pad)
    d_rows, d_w, again = _wide(torch.full((n_rows, H), MARK, dtype=dt), pad), torch.full((T, k), MARK, device="cuda"), torch.zeros((T, k), device="cuda")
    moe.moe_combine_rows_backward(dy, rows, w, inv, d_rows, d_w)
    prod = mine * dy.double()[:, None, :]
    kept = rows.clone()
    moe.moe_combine_rows_backward(dy, rows, w, inv, rows, again)
    torch.cuda.synchronize()
    _close(d_w, prod.sum(2), H * P.U * prod.abs().sum(2))  # H fused multiply-adds and additions at most
    del prod, mine
    at, (tok, j) = inv.long().view(T, k)[live], torch.nonzero(live, as_tuple=True)
    ref = w.double()[tok, j][:, None] * dy.double()[tok]
    _close(d_rows[at], ref, P.stored(ref, P.U * ref.abs(), dt))
    free = torch.ones(n_rows, dtype=torch.bool, device="cuda")
    free[at] = False
    assert (d_rows[free] == MARK).all() and torch.equal(rows[free], kept[free])
    assert torch.equal(rows[at], d_rows[at]) and torch.equal(again, d_w)
    for t in (x, rows, y, dx, d_rows) if pad else ():
        assert torch.isnan(t._base[:, H:].float()).all()


@pytest.mark.parametrize("T,k,E,H", [(33, 20, 64, 2049), (70, 9, 64, 1030), (7, 32, 40, 1500), (129, 8, 16, 1025), (300, 17, 24, 4099)])
@pytest.mark.parametrize("dt,ydt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("drop,pad,fewer", [(0.0, 0, 0), (0.3, 3, 5)])
def test_token_in_a_workgroup(T, k, E, H, dt, ydt, drop, pad, fewer):
    _all_calls(T, k, E, H, dt, ydt, drop, pad, fewer)


@pytest.mark.parametrize("T,k,H,dt", [(2100, 4, 1030, F32), (2100, 4, 1003, F32), (4100, 8, 1030, F32), (4200, 8, 1003, F32),
                                      (4200, 8, 2049, BF16), (17100, 8, 1003, BF16)])
def test_rows_past_the_caches(T, k, H, dt):
    """Rows of more than 32 MB, read past the caches, and of more than 128 MB, written past them, too; in waves and in workgroups."""
    size = T * k * H * (2 if dt is BF16 else 4)
    assert size > (128 << 20 if k == 8 else 32 << 20)
    _all_calls(T, k, 60, H, dt, dt, 0.0, 1, 0)
    torch.cuda.empty_cache()
