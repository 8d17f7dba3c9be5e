"""moe_block_norm against its plain form in 64 bits."""
import pytest
import torch

import plain_ops as P
from routed_expert_ffn_layer_amd import moe

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
N, R, L = moe.MOE_NORM_NONE, moe.MOE_NORM_RMS, moe.MOE_NORM_LAYER


def _run(T, H, bdt=BF16, rdt=BF16, xdt=BF16, post=R, pre=R, gate="channel", gdt=F32, pads=(0, 0, 0, 0, 0), seed=1, eps=1e-6,
         biases=True, make=None, in_place=False, no_block=False, no_res=False, scales=(0.7, 0.9)):
    """One call against the plain form; make(T, H) gives block and res in f64."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    block, res = make(T, H) if make else (n(T, H), 3 * n(T, H) + 0.5)
    norms = {}
    for name, kind in (("post", post), ("pre", pre)):
        norms[name] = (kind, 1 + 0.1 * n(H), 0.1 * n(H) if biases else None) if kind else None
    gv = None if gate == "none" else (0.5 * n(H) if gate == "channel" else 0.5 * n(T, H)).to(gdt)

    def rows(v, dt, pad):  # rows pad columns apart, NaN between them
        wide = torch.full((max(T, 1), H + pad), float("nan"), dtype=dt, device="cuda")
        wide[:T, :H] = v.to(dt)
        return wide[:T, :H]

    b = None if no_block else rows(block, bdt, pads[0])
    r = None if no_res else rows(res, rdt, pads[1])
    gd = None if gv is None else (gv.cuda() if gv.dim() == 1 else rows(gv, gdt, pads[4]))
    on = lambda m: None if m is None else (m[0], *(v if v is None else v.cuda() for v in m[1:]))  # noqa: E731
    ref_r, ref_x = P.block_norm(None if no_block else b.cpu(), norms["post"], gv, scales[0], None if no_res else r.cpu(),
                                scales[1], norms["pre"], eps)
    out = r if in_place else rows(torch.zeros(T, H), rdt, pads[2])
    x = b if in_place else rows(torch.zeros(T, H), xdt, pads[3])
    moe.moe_block_norm(b, on(norms["post"]), gd, scales[0], r, scales[1], on(norms["pre"]), eps, out, x)
    torch.cuda.synchronize()
    P.check(out, ref_r[0], P.stored(*ref_r, rdt), "res_out")
    P.check(x, ref_x[0], P.stored(*ref_x, x.dtype), "x")
    for v in (out, x):  # nothing between the rows is written
        pad = v._base
        if pad is not None and pad.dim() == 2 and pad.shape[1] > H and not in_place:
            assert torch.isnan(pad[:T, H:].float()).all()


@pytest.mark.parametrize("H", [1, 2, 7, 8, 9, 63, 64, 511, 512, 513, 520, 1000, 2048, 2085, 4096, 8191, 8192, 8200, 16384, 16392, 32767, 32768])
def test_widths(H):
    for kind in (R, L):
        _run(5, H, post=kind, pre=kind, seed=H)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 64, 257])
@pytest.mark.parametrize("H", [96, 1024])
def test_tokens(T, H):
    _run(T, H, seed=T)


@pytest.mark.parametrize("bdt", [BF16, F32])
@pytest.mark.parametrize("rdt", [BF16, F32])
@pytest.mark.parametrize("xdt", [BF16, F32])
@pytest.mark.parametrize("gate,gdt", [("channel", F32), ("token", BF16), ("token", F32), ("channel", BF16)])
def test_types(bdt, rdt, xdt, gate, gdt):
    _run(3, 200, bdt, rdt, xdt, gate=gate, gdt=gdt)
    _run(3, 1003, bdt, rdt, xdt, L, L, gate=gate, gdt=gdt)


@pytest.mark.parametrize("post", [N, R, L])
@pytest.mark.parametrize("pre", [N, R, L])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_kinds(post, pre, gate):
    _run(6, 777, F32, F32, F32, post, pre, gate)
    _run(6, 776, BF16, BF16, BF16, post, pre, gate, biases=False)


@pytest.mark.parametrize("pads", [(1, 0, 0, 0, 0), (0, 3, 0, 0, 5), (0, 0, 1, 7, 8), (5, 1, 3, 8, 2), (8, 16, 24, 32, 40)])
@pytest.mark.parametrize("H", [100, 1027])
def test_strides(pads, H):
    _run(7, H, gate="token", gdt=BF16, pads=pads)
    _run(7, H, F32, F32, F32, L, L, gate="token", pads=pads)


def test_in_place():
    _run(9, 640, in_place=True)
    _run(9, 4097, F32, F32, F32, L, L, in_place=True)


def test_without_block_or_residual():
    _run(4, 512, post=N, gate="none", no_block=True, scales=(5.0, 1.0))
    _run(4, 520, pre=L, no_res=True, scales=(0.25, float("nan")))


def test_outputs_that_are_not_wanted():
    b, r = torch.randn(3, 264, device="cuda"), torch.randn(3, 264, device="cuda")
    both, x = torch.empty_like(r), torch.empty_like(b)
    moe.moe_block_norm(b, None, None, 1.0, r, 1.0, (R, None), 1e-6, both, x)
    one, y = torch.empty_like(r), torch.empty_like(b)
    moe.moe_block_norm(b, None, None, 1.0, r, 1.0, None, 1e-6, one, None)
    moe.moe_block_norm(b, None, None, 1.0, r, 1.0, (R, None), 1e-6, None, y)
    torch.cuda.synchronize()
    assert torch.equal(one, both) and torch.equal(x, y)


def test_no_tokens():
    e = torch.empty((0, 64), device="cuda")
    moe.moe_block_norm(e, (R, None), None, 1.0, e, 1.0, (R, None), 1e-6, e, e)


@pytest.mark.parametrize("H", [48, 600, 9000])
@pytest.mark.parametrize("kind", [R, L])
def test_sums_beyond_f32(H, kind):
    """Elements whose squares, or whose sums, leave the f32 range; tiny ones without an eps."""
    g = torch.Generator().manual_seed(H)
    for size in (1e25, 3e37, 1e-25, 2.0 ** -130):
        make = lambda T, H: ((torch.randn(T, H, generator=g) * size).clamp(-3e38, 3e38), torch.zeros(T, H))  # noqa: B023, E731
        _run(3, H, F32, F32, F32, post=kind, pre=N, gate="none", make=make, eps=0.0 if size < 1 else 1e-6, no_res=True, biases=False)


def test_rows_of_one_huge_element():
    v = torch.zeros(2, 1000)
    v[0, 7], v[1, 999] = 3.0e38, -2.5e38
    _run(2, 1000, F32, F32, F32, pre=N, gate="none", make=lambda T, H: (v, v), no_res=True)


def test_large_offset():
    """A layer norm of values 1000 apart from 0 by a deviation of 1."""
    g = torch.Generator().manual_seed(3)
    _run(4, 3001, F32, F32, F32, L, N, "none", make=lambda T, H: (1000 + torch.randn(T, H, generator=g), torch.zeros(T, H)))


def test_equal_values():
    """Variance 0: eps alone divides."""
    v = torch.full((2, 515), 0.1)
    _run(2, 515, F32, F32, F32, L, N, "none", make=lambda T, H: (v, v))


def test_infinite_and_nan_rows_stay_alone():
    g = torch.Generator().manual_seed(9)
    b, r = torch.randn(6, 300, generator=g), torch.randn(6, 300, generator=g)
    b[1, 5], b[3, 299] = float("nan"), float("inf")
    out, x = torch.empty(6, 300, device="cuda"), torch.empty(6, 300, device="cuda")
    moe.moe_block_norm(b.cuda(), (R, None), None, 1.0, r.cuda(), 1.0, (L, None), 1e-6, out, x)
    torch.cuda.synchronize()
    fine = [0, 2, 4, 5]
    (ref, tol), (rx, tx) = P.block_norm(b, (R, None, None), None, 1.0, r, 1.0, (L, None, None), 1e-6)
    P.check(out[fine], ref[fine], P.stored(ref, tol, F32)[fine])
    P.check(x[fine], rx[fine], P.stored(rx, tx, F32)[fine])
    assert torch.isnan(out[1]).all() and torch.isnan(x[[1, 3]]).all() and torch.isnan(out[3, 299])
    assert torch.equal(out[3, :299].cpu(), r[3, :299])  # finite over infinite is 0


def test_other_stream_and_graph():
    g = torch.Generator().manual_seed(4)
    b, r = torch.randn(16, 1000, generator=g).cuda(), torch.randn(16, 1000, generator=g).cuda()
    want, wx = torch.empty_like(r), torch.empty_like(b)
    call = lambda o, x: moe.moe_block_norm(b, (R, None), None, 0.5, r, 1.0, (L, None), 1e-6, o, x)  # noqa: E731
    call(want, wx)
    out, x = torch.zeros_like(r), torch.zeros_like(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call(out, x)
        side.synchronize()
        assert torch.equal(out, want)
        with torch.cuda.graph(graph, stream=side):
            call(out, x)
    for i in range(3):
        b.mul_(-1.0)
        call(want, wx)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(x, wx)
