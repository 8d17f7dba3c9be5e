"""Rows past 4 GiB of their buffer, in bytes and in elements: every operator that takes a stride or many rows.
(One buffer of 20 GiB serves all; only the rows in use are ever touched.)"""
import pytest
import torch

import plain_ops as P
from routed_expert_ffn_layer_amd import moe

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def far():
    """rows, width, type -> a matrix whose last row begins past 2^32 elements (f32: past 2^34 bytes)."""
    buf = torch.empty(20 << 30, dtype=torch.uint8, device="cuda")

    def make(rows, width, dt):
        flat = buf.view(dt)
        return flat.as_strided((rows, width), ((flat.numel() - 4096) // (rows - 1) // 8 * 8, 1))

    yield make
    del buf
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_norm(far, dt):
    g = torch.Generator().manual_seed(1)
    b, r = torch.randn(5, 777, generator=g).to(dt), torch.randn(5, 777, generator=g).to(dt)
    rows = far(5, 777, dt)
    rows.copy_(b)
    out, x = torch.empty((5, 777), dtype=dt, device="cuda"), rows
    moe.moe_block_norm(rows, (1, None), None, 1.0, r.cuda(), 1.0, (1, None), 1e-6, out, x)
    torch.cuda.synchronize()
    ref, nxt = P.block_norm(b, (1, None, None), None, 1.0, r, 1.0, (1, None, None), 1e-6)
    P.check(out, ref[0], P.stored(*ref, dt))
    P.check(x, nxt[0], P.stored(*nxt, dt))


@pytest.mark.parametrize("T", [2, 40, 300])
def test_linear_results(far, T):
    g = torch.Generator().manual_seed(T)
    x, w = torch.randint(-4, 5, (T, 64), generator=g).to(BF16), torch.randint(-4, 5, (50, 64), generator=g).to(BF16)
    y = far(T, 50, F32)
    y.fill_(3.0)
    moe.moe_linear(w.cuda(), x.cuda(), None, 0, y, y)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu().double(), x.double() @ w.double().t() + 3)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("dt,N", [(BF16, 9000), (F32, 4500)])
def test_linear_weights(T, dt, N):
    """Weight rows 2^20 elements apart, 17.6 GiB of them."""
    buf = torch.empty(N << 20, dtype=dt, device="cuda")
    w = buf.as_strided((N, 24), (1 << 20, 1))
    g = torch.Generator(device="cuda").manual_seed(T)
    w.copy_(torch.randint(-4, 5, (N, 24), generator=g, device="cuda"))
    x = torch.randint(-4, 5, (T, 24), generator=g, device="cuda").to(dt)
    y = torch.empty((T, N), device="cuda")
    moe.moe_linear(w, x, None, 0, None, y)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu().double(), x.cpu().double() @ w.cpu().double().t())
    del buf, w
    torch.cuda.empty_cache()


def test_sorted_rows_beyond_4_gib():
    """75000 rows of 32768: places past 2^31 elements and 4 GiB, both ways and the gradients."""
    T, k, E, H = 9375, 8, 16, 32768
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randn((T, E), generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    x = torch.randn((T, 64), generator=g, device="cuda").to(BF16).repeat(1, H // 64)
    x += torch.arange(H, device="cuda").to(BF16)[None, :] % 7
    i32 = dict(dtype=torch.int32, device="cuda")
    order = [torch.empty(n, **i32) for n in (E, E + 1, T * k, T * k)]
    rows = torch.empty((T * k, H), dtype=BF16, device="cuda")
    ws = torch.empty(moe.moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda")
    moe.moe_dispatch(x, ids, E, *order, rows, ws)
    torch.cuda.synchronize()
    for a, b in zip(order, P.order(ids.cpu(), E)):
        assert torch.equal(a.cpu(), b)
    tok = order[2].long() // k
    for lo in range(0, T * k, 8192):
        assert torch.equal(rows[lo:lo + 8192], x[tok[lo:lo + 8192]])
    w = torch.full((T, k), 0.125, device="cuda")
    y = torch.empty_like(x)
    moe.moe_combine_rows(rows, w, order[3], y)
    assert torch.equal(y, x)  # 8 times an eighth of the same row, every partial sum a multiple of an eighth of a bf16: exact in f32
    d_w = torch.empty((T, k), device="cuda")
    moe.moe_combine_rows_backward(x, rows, w, order[3], rows, d_w)  # in place
    torch.cuda.synchronize()
    for lo in range(0, T * k, 8192):
        assert torch.equal(rows[lo:lo + 8192], x[tok[lo:lo + 8192]] * 0.125)
    ref, mag = (x.double() ** 2).sum(1), (x.double() ** 2).sum(1)
    P.check(d_w, ref[:, None].expand(T, k), (H * P.U * mag)[:, None].expand(T, k))
    dx = torch.empty_like(x)
    moe.moe_dispatch_backward(rows, order[3], k, dx)
    torch.cuda.synchronize()
    assert torch.equal(dx, x)
    del rows, x
    torch.cuda.empty_cache()
