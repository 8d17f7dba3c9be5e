"""Calls of the block norm, the linear product and the sorted tokens that are refused: by the C ABI before
any device work, and by the binding for tensors that the library would read as other data (no GPU needed)."""
import ctypes

import pytest
import torch

from routed_expert_ffn_layer_amd import moe

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
MB = 1 << 20


def _p(mb, off=0):
    return ctypes.c_void_p(mb * MB + off)


def _norm(**change):
    a = dict(block=_p(16), bdt=1, b_ld=64, post=1, post_w=_p(1), post_b=None, gate=_p(2), gdt=0, gate_ld=0, bs=1.0, res=_p(17),
             r_ld=64, rs=1.0, pre=2, pre_w=_p(3), pre_b=_p(4), eps=1e-6, T=4, H=64, out=_p(18), rdt=1, o_ld=64, x=_p(19), xdt=1,
             x_ld=64)
    a.update(change)
    return moe.lib().moe_block_norm(*a.values(), None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(T=(1 << 21) + 1), dict(H=0), dict(H=-8), dict(post=3), dict(post=-1), dict(pre=3), dict(bdt=2), dict(rdt=4),
    dict(xdt=-1), dict(gdt=7), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(block=None, res=None), dict(out=None, x=None), dict(block=None), dict(post=0), dict(x=None), dict(pre=0),
    dict(b_ld=63), dict(r_ld=0), dict(gate_ld=32), dict(o_ld=63), dict(x_ld=-64), dict(block=_p(16, 8)), dict(x=_p(19, 2)),
    dict(post_w=_p(1, 4)), dict(pre_b=_p(4, 8)), dict(out=_p(19)), dict(out=_p(19, 128)), dict(x=_p(16, 16)), dict(x=_p(16), xdt=0),
    dict(x=_p(16), x_ld=72), dict(out=_p(17, 128)), dict(out=_p(2)), dict(x=_p(1)), dict(out=_p(3), o_ld=80)])
def test_norm(change):
    assert _norm(**change) == moe.MOE_EINVAL


def test_norm_too_wide_and_no_tokens():
    assert _norm(H=32769, b_ld=40000) == moe.MOE_EUNSUPPORTED
    assert _norm(T=0, block=None, res=None, out=None, x=None, gate=None) == moe.MOE_OK


def _linear(**change):
    a = dict(wdt=1, w=_p(16), w_ld=64, N=32, K=64, x=_p(32), x_ld=64, T=4, bias=_p(1), act=0, res=_p(40), rdt=1, r_ld=32, y=_p(48),
             ydt=1, y_ld=32)
    a.update(change)
    return moe.lib().moe_linear(*a.values(), None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(T=(1 << 22) + 1), dict(N=0), dict(N=-1), dict(N=(1 << 22) + 1), dict(T=1 << 22, N=1 << 14), dict(K=0), dict(K=-8),
    dict(K=4), dict(K=60), dict(K=(1 << 20) + 8), dict(wdt=0, K=62, w_ld=64), dict(act=5), dict(act=-1), dict(ydt=2), dict(rdt=3),
    dict(w_ld=56), dict(w_ld=68), dict(x_ld=63), dict(x_ld=(1 << 21) + 8), dict(w_ld=(1 << 21) + 8), dict(y_ld=31), dict(r_ld=16), dict(w=None),
    dict(x=None), dict(y=None), dict(w=_p(16, 2)), dict(x=_p(32, 8)), dict(y=_p(48, 4)), dict(res=_p(40, 2)), dict(bias=_p(1, 4)), dict(y=_p(16)),
    dict(y=_p(32, 64)), dict(y=_p(1)), dict(y=_p(40), ydt=0), dict(y=_p(40), y_ld=40), dict(y=_p(40, 16))])
def test_linear(change):
    assert _linear(**change) == moe.MOE_EINVAL


def test_linear_other_weights_and_no_tokens():
    assert _linear(wdt=moe.MOE_MXFP4) == moe.MOE_EUNSUPPORTED
    assert _linear(wdt=moe.MOE_INT4) == moe.MOE_EUNSUPPORTED
    assert _linear(T=0, x=None, y=None, res=None) == moe.MOE_OK


def _dispatch(**change):  # more pairs than are placed without a workspace
    a = dict(x=_p(16), xdt=1, x_ld=64, ids=_p(1), T=20000, k=2, E=8, H=64, counts=_p(2), offsets=_p(3), rows_order=_p(4), inv=_p(5),
             rows=_p(32), rows_ld=64, n_rows=40000, ws=_p(6), ws_bytes=1 << 20)
    a.update(change)
    return moe.lib().moe_dispatch(*a.values(), None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(T=(1 << 21) + 1), dict(k=0), dict(k=9), dict(k=33, E=64), dict(E=0), dict(E=1025), dict(H=0), dict(H=(1 << 24) + 1, x_ld=1 << 25, rows_ld=1 << 25),
    dict(xdt=2), dict(x_ld=63), dict(rows_ld=32), dict(n_rows=-1), dict(x=None), dict(ids=None), dict(counts=None), dict(offsets=None),
    dict(rows_order=None), dict(inv=None), dict(rows=None), dict(ws=None), dict(x=_p(16, 8)), dict(rows=_p(32, 2)), dict(ids=_p(1, 4)),
    dict(rows=_p(16)), dict(rows=_p(16, 128))])
def test_dispatch(change):
    assert _dispatch(**change) == moe.MOE_EINVAL


def test_dispatch_workspace():
    n = moe.moe_dispatch_workspace(20000, 2, 8)
    assert n > 0 and _dispatch(ws_bytes=n - 1) == moe.MOE_ECAPACITY
    assert moe.moe_dispatch_workspace(10, 2, 8) == moe.moe_dispatch_workspace(4096, 2, 8) == 0
    assert moe.moe_dispatch_workspace(10, 9, 8) == moe.moe_dispatch_workspace(-1, 1, 8) == moe.moe_dispatch_workspace(1 << 22, 1, 8) == 0


def _combine(**change):
    a = dict(rows=_p(16), rdt=1, rows_ld=64, n_rows=8, w=_p(1), inv=_p(2), T=4, k=2, H=64, y=_p(17), ydt=1, y_ld=64)
    a.update(change)
    return moe.lib().moe_combine_rows(*a.values(), None)


def _combine_back(**change):
    a = dict(dy=_p(15), ydt=1, dy_ld=64, rows=_p(16), rdt=1, rows_ld=64, n_rows=8, w=_p(1), inv=_p(2), T=4, k=2, H=64, d_rows=_p(17), dr_ld=64,
             d_w=_p(3))
    a.update(change)
    return moe.lib().moe_combine_rows_backward(*a.values(), None)


@pytest.mark.parametrize("change", [dict(T=-1), dict(T=(1 << 21) + 1), dict(k=0), dict(k=33), dict(H=0), dict(n_rows=-1), dict(rdt=2), dict(ydt=4), dict(rows=None),
                                    dict(w=None), dict(inv=None), dict(rows_ld=63), dict(rows=_p(16, 8)), dict(w=_p(1, 4)), dict(inv=_p(2, 8))])
def test_combine(change):
    assert _combine(**change) == moe.MOE_EINVAL
    assert _combine_back(**change) == moe.MOE_EINVAL


@pytest.mark.parametrize("change", [dict(y=None), dict(y_ld=8), dict(y=_p(17, 4)), dict(y=_p(16)), dict(y=_p(16, 256))])
def test_combine_result(change):
    assert _combine(**change) == moe.MOE_EINVAL


@pytest.mark.parametrize("change", [dict(dy=None), dict(dy_ld=8), dict(dy=_p(15, 4)), dict(d_rows=None), dict(dr_ld=8), dict(d_rows=_p(15)), dict(d_rows=_p(16, 128)),
                                    dict(d_rows=_p(16), dr_ld=72), dict(d_w=None), dict(d_w=_p(3, 4)), dict(d_w=_p(1))])
def test_combine_gradient(change):
    assert _combine_back(**change) == moe.MOE_EINVAL


def test_dispatch_gradient_and_gate():
    L = moe.lib()
    ok = [_p(16), 1, 64, 8, _p(2), 4, 2, 64, _p(17), 1, 64]
    for i, bad in ((0, None), (1, 2), (2, 63), (3, -1), (4, None), (5, -1), (6, 0), (7, 0), (8, None), (8, _p(16)), (9, 3), (10, 63)):
        assert L.moe_dispatch_backward(*ok[:i], bad, *ok[i + 1:], None) == moe.MOE_EINVAL
    ok = [_p(1), _p(2), _p(3), 4, 8, 2, _p(4)]
    for i, bad in ((0, None), (1, None), (2, _p(3, 4)), (3, -1), (3, (1 << 21) + 1), (4, 0), (4, 1025), (5, 0), (5, 9), (6, None)):
        assert L.moe_gate_backward(*ok[:i], bad, *ok[i + 1:], None) == moe.MOE_EINVAL


# ---------------------------------------------------------------------------
# The binding
# ---------------------------------------------------------------------------
T, H, N, K, E, TOPK = 6, 32, 24, 16, 8, 2


def _refused(what, call):
    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.status == moe.MOE_EINVAL and what in str(e.value), str(e.value)


@pytest.mark.parametrize("what,change", [
    ("w", dict(w=torch.zeros((N, K), dtype=torch.float16))), ("x", dict(x=torch.zeros((T, K)))), ("x", dict(x=torch.zeros((K, T), dtype=BF16).t())),
    ("x", dict(x=torch.zeros((T, K + 8), dtype=BF16))), ("w", dict(w=torch.zeros(N, dtype=BF16))), ("x", dict(x=torch.zeros((1, T, K), dtype=BF16))),
    ("bias", dict(bias=torch.zeros(N, dtype=BF16))), ("bias", dict(bias=torch.zeros(N + 1))), ("bias", dict(bias=torch.zeros(1).expand(N))),
    ("res", dict(res=torch.zeros((T, N), dtype=torch.float64))), ("res", dict(res=torch.zeros((1, N)))), ("res", dict(res=torch.zeros((N, T)).t())),
    ("y", dict(y=torch.zeros((T, N), dtype=torch.int16))), ("y", dict(y=torch.zeros((T + 1, N)))), ("y", dict(y=torch.zeros((N, T)).t()))])
def test_linear_tensors(what, change):
    a = dict(w=torch.zeros((N, K), dtype=BF16), x=torch.zeros((T, K), dtype=BF16), bias=None, act=0, res=None, y=torch.zeros((T, N)))
    a.update(change)
    _refused(what, lambda: moe.moe_linear(*a.values()))


@pytest.mark.parametrize("what,change", [
    ("neither", dict(block=None, res=None)), ("neither", dict(out=None, x=None)), ("block", dict(block=torch.zeros((T, H), dtype=torch.float16))),
    ("matrix", dict(block=torch.zeros(H))), ("res", dict(res=torch.zeros((T + 1, H)))), ("res_out", dict(out=torch.zeros((T, H), dtype=BF16))),
    ("x", dict(x=torch.zeros((T, 2 * H))[:, ::2])), ("gate", dict(gate=torch.zeros((H, H)))), ("gate", dict(gate=torch.zeros(H + 1))),
    ("gate", dict(gate=torch.zeros(2 * H)[::2])), ("gate", dict(gate=torch.zeros(H, dtype=torch.float16))),
    ("post norm's weight", dict(post=(1, torch.zeros(H, dtype=BF16)))), ("post norm's bias", dict(post=(2, torch.zeros(H), torch.zeros(1)))),
    ("pre norm's weight", dict(pre=(1, torch.zeros(1).expand(H)))), ("pre norm's bias", dict(pre=(2, None, torch.zeros((H, 2))[:, 0])))])
def test_norm_tensors(what, change):
    a = dict(block=torch.zeros((T, H)), post=None, gate=None, bs=1.0, res=torch.zeros((T, H)), rs=1.0, pre=(1, None), eps=1e-6, out=torch.zeros((T, H)),
             x=torch.zeros((T, H)))
    a.update(change)
    _refused(what, lambda: moe.moe_block_norm(*a.values()))


def _sorted(**change):
    n = T * TOPK
    a = dict(x=torch.zeros((T, H)), ids=torch.zeros((T, TOPK), dtype=I32), E=E, counts=torch.zeros(E, dtype=I32), offsets=torch.zeros(E + 1, dtype=I32),
             order=torch.zeros(n, dtype=I32), inv=torch.zeros(n, dtype=I32), rows=torch.zeros((n, H)), ws=torch.zeros(16, dtype=U8))
    a.update(change)
    moe.moe_dispatch(*a.values())


@pytest.mark.parametrize("what,change", [
    ("x", dict(x=torch.zeros((T, H), dtype=torch.float16))), ("rows", dict(rows=torch.zeros((T * TOPK, H), dtype=BF16))),
    ("rows", dict(rows=torch.zeros((T * TOPK, H + 1)))), ("topk_ids", dict(ids=torch.zeros((T, TOPK), dtype=torch.int64))),
    ("topk_ids", dict(ids=torch.zeros((T, 2 * TOPK), dtype=I32)[:, ::2])), ("topk_ids", dict(ids=torch.zeros((T + 1, TOPK), dtype=I32))),
    ("counts", dict(counts=torch.zeros(E + 1, dtype=I32))), ("offsets", dict(offsets=torch.zeros(E, dtype=I32))), ("sorted_rows", dict(order=torch.zeros(T, dtype=I32))),
    ("inv_rows", dict(inv=torch.zeros(T * TOPK, dtype=torch.int64))), ("workspace", dict(ws=torch.zeros(1, dtype=U8).expand(100))), ("matrix", dict(ids=torch.zeros(T, dtype=I32)))])
def test_dispatch_tensors(what, change):
    _refused(what, lambda: _sorted(**change))


@pytest.mark.parametrize("what,change", [
    ("rows", dict(rows=torch.zeros((4, H + 1)))), ("topk_w", dict(w=torch.zeros((T, TOPK), dtype=BF16))), ("inv_rows", dict(inv=torch.zeros(3, dtype=I32))),
    ("inv_rows", dict(inv=None)), ("y", dict(y=torch.zeros((T + 1, H)))), ("y", dict(y=torch.zeros((T, H), dtype=torch.float16)))])
def test_combine_tensors(what, change):
    a = dict(rows=torch.zeros((4, H)), w=torch.zeros((T, TOPK)), inv=torch.zeros(T * TOPK, dtype=I32), y=torch.zeros((T, H)))
    a.update(change)
    _refused(what, lambda: moe.moe_combine_rows(*a.values()))
    if what != "y":
        _refused(what, lambda: moe.moe_combine_rows_backward(a["y"], a["rows"], a["w"], a["inv"], torch.zeros((4, H)), torch.zeros((T, TOPK))))


def test_vectors_and_none_in_place_of_matrices():
    v, inv, w = torch.zeros(H), torch.zeros(T * TOPK, dtype=I32), torch.zeros((T, TOPK))
    m = torch.zeros((T, H))
    for call in (lambda: moe.moe_combine_rows(v, w, inv, m), lambda: moe.moe_combine_rows(m, w.reshape(-1), inv, m), lambda: moe.moe_combine_rows(m, None, inv, m),
                 lambda: moe.moe_combine_rows(m, w, inv, None), lambda: moe.moe_dispatch_backward(v, inv, TOPK, m), lambda: moe.moe_dispatch_backward(m, inv, TOPK, v),
                 lambda: moe.moe_combine_rows_backward(m, v, w, inv, m, w), lambda: moe.moe_gate_backward(inv, w.reshape(-1), w, m),
                 lambda: moe.moe_linear(None, m, None, 0, None, m), lambda: moe.moe_linear(m, None, None, 0, None, m)):
        _refused("matrix", call)


def test_rows_too_far_apart():
    far = (1 << 36) + 8
    assert _norm(b_ld=far) == _norm(o_ld=far) == _linear(y_ld=far) == _linear(r_ld=far) == moe.MOE_EINVAL
    assert _dispatch(x_ld=far) == _dispatch(rows_ld=far) == _combine(rows_ld=far) == _combine_back(dr_ld=far) == moe.MOE_EINVAL


def test_gradient_tensors():
    inv, w = torch.zeros(T * TOPK, dtype=I32), torch.zeros((T, TOPK))
    back = lambda **c: moe.moe_combine_rows_backward(*dict(dict(dy=torch.zeros((T, H)), rows=torch.zeros((4, H)), w=w, inv=inv, d_rows=torch.zeros((4, H)), d_w=w.clone()), **c).values())  # noqa: E731
    _refused("d_rows", lambda: back(d_rows=torch.zeros((4, H), dtype=BF16)))
    _refused("d_rows", lambda: back(d_rows=torch.zeros((5, H))))
    _refused("d_topk_w", lambda: back(d_w=torch.zeros((T, TOPK), dtype=BF16)))
    _refused("dy", lambda: back(dy=torch.zeros((T - 1, H))))
    _refused("inv_rows", lambda: moe.moe_dispatch_backward(torch.zeros((4, H)), inv, TOPK + 1, torch.zeros((T, H))))
    _refused("d_rows", lambda: moe.moe_dispatch_backward(torch.zeros((4, H - 1)), inv, TOPK, torch.zeros((T, H))))
    _refused("d_logits", lambda: moe.moe_gate_backward(torch.zeros((T, TOPK), dtype=I32), w, w, torch.zeros((T, E), dtype=BF16)))
    _refused("d_topk_w", lambda: moe.moe_gate_backward(torch.zeros((T, TOPK), dtype=I32), w, torch.zeros((T, 1)), torch.zeros((T, E))))


# ---------------------------------------------------------------------------
# Results on each other or on what is still read
@pytest.mark.parametrize("change", [
    dict(counts=_p(3)), dict(counts=_p(1)), dict(offsets=_p(2, 16)), dict(rows_order=_p(5)), dict(inv=_p(4, 16)), dict(rows_order=_p(1)),
    dict(inv=_p(1, 159984)), dict(ws=_p(1)), dict(ws=_p(4)), dict(ws=_p(5, 64)), dict(ws=_p(2)), dict(rows=_p(1)), dict(rows=_p(5)),
    dict(rows=_p(6)), dict(counts=_p(16)), dict(ws=_p(16)), dict(inv=_p(32, 128)), dict(rows_order=_p(16))])
def test_dispatch_results_apart(change):
    assert _dispatch(**change) == moe.MOE_EINVAL


def test_combine_results_apart():
    assert _combine(y=_p(1)) == _combine(y=_p(2)) == _combine(w=_p(17, 16)) == moe.MOE_EINVAL
    for change in (dict(d_w=_p(2)), dict(d_w=_p(15)), dict(d_w=_p(16)), dict(d_w=_p(17)), dict(d_w=_p(1, 16)), dict(d_rows=_p(1)),
                   dict(d_rows=_p(2)), dict(d_rows=_p(3))):
        assert _combine_back(**change) == moe.MOE_EINVAL
    ok = [_p(1), _p(2), _p(3), 4, 8, 2, _p(4)]
    for on in (1, 2, 3):
        assert moe.lib().moe_gate_backward(*ok[:6], _p(on), None) == moe.MOE_EINVAL
