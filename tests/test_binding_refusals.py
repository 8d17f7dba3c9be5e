"""Tensors that the Python binding of the few-token operators refuses because the library,
which sees addresses only, would read them as other data or past their end (runs without a GPU:
these checks come before any look at a device)."""
import pytest
import torch

from routed_expert_ffn_layer_amd import moe

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
N, K, T = 32, 64, 3


def _refused(what, call, status=moe.MOE_EINVAL):
    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.status == status and what in str(e.value), str(e.value)


def _packed():
    return torch.zeros(moe.moe_w4_bytes(moe.MOE_INT4, N, K, 64), dtype=U8)


@pytest.mark.parametrize("what,change", [
    ("x", dict(x=torch.zeros((T, K), dtype=F32))), ("x", dict(x=torch.zeros((T, K), dtype=torch.float16))),
    ("x", dict(x=torch.zeros((T, K), dtype=U8))),
    ("bias", dict(bias=torch.zeros(N, dtype=BF16))), ("bias", dict(bias=torch.zeros(N, dtype=torch.float64))),
    ("bias", dict(bias=torch.zeros(N - 1))), ("bias", dict(bias=torch.zeros(2 * N)[::2])),
    ("bias", dict(bias=torch.zeros((N, 1)))), ("bias", dict(bias=torch.zeros(1).expand(N))),
    ("w", dict(w=_packed()[:-1])), ("w", dict(w=torch.zeros(2 * _packed().numel(), dtype=U8)[::2])),
    ("w", dict(w=torch.zeros(0, dtype=U8)))])
def test_linear(what, change):
    a = dict(w=_packed(), x=torch.zeros((T, K), dtype=BF16), bias=None, y=torch.zeros((T, N)))
    a.update(change)
    _refused(what, lambda: moe.moe_w4_linear(moe.MOE_INT4, a["w"], N, K, 64, a["x"], a["bias"], a["y"]))


TD, H, I, E, TOPK = 4, 64, 32, 8, 2


def _layer(**change):
    eb = moe.moe_expert_bytes(moe.MOE_BF16, H, I)
    a = dict(pool=torch.zeros((E, eb), dtype=U8), slots=torch.zeros(E, dtype=torch.int32), shared=None, ish=0,
             x=torch.zeros((TD, H), dtype=BF16), logits=torch.zeros((TD, E)), ids=torch.zeros((TD, TOPK), dtype=torch.int32),
             w=torch.zeros((TD, TOPK)), y=torch.zeros((TD, H), dtype=BF16), ydt=moe.MOE_BF16,
             ws=torch.zeros(moe.moe_layer_decode_workspace(TD, TOPK, E, H, I, 32, moe.MOE_BF16), dtype=U8))
    a.update(change)
    moe.moe_layer_decode(moe.MOE_BF16, a["pool"], eb, a["slots"], a["shared"], a["ish"], a["x"], a["logits"], TD, TOPK, E, H,
                         I, a["ids"], a["w"], a["y"], a["ydt"], a["ws"])


@pytest.mark.parametrize("what,change", [
    ("x", dict(x=torch.zeros((TD, H)))), ("x", dict(x=torch.zeros((TD, H), dtype=torch.float16))),
    ("x", dict(x=torch.zeros((TD - 1, H), dtype=BF16))), ("x", dict(x=torch.zeros((TD, 2 * H), dtype=BF16)[:, :H])),
    ("x", dict(x=torch.zeros((H, TD), dtype=BF16).t())), ("x", dict(x=torch.zeros((TD, 2 * H), dtype=BF16))),
    ("x", dict(x=torch.zeros((1, H), dtype=BF16).expand(TD, H))),
    ("logits", dict(logits=torch.zeros((TD, E), dtype=BF16))), ("logits", dict(logits=torch.zeros((TD, E + 1))[:, :E])),
    ("logits", dict(logits=torch.zeros((TD - 1, E)))),
    ("topk_ids", dict(ids=torch.zeros((TD, TOPK), dtype=torch.int64))), ("topk_ids", dict(ids=torch.zeros((TD, 1), dtype=torch.int32))),
    ("topk_ids", dict(logits=None, ids=torch.zeros((TD, TOPK), dtype=torch.int64))),
    ("topk_w", dict(w=torch.zeros((TD, TOPK), dtype=BF16))), ("topk_w", dict(w=torch.zeros((1, TOPK)))),
    ("topk_w", dict(logits=None, w=torch.zeros((TD, TOPK), dtype=torch.float64))),
    ("slot_of_expert", dict(slots=torch.zeros(E, dtype=torch.int64))), ("slot_of_expert", dict(slots=torch.zeros(E - 1, dtype=torch.int32))),
    ("slot_of_expert", dict(slots=torch.zeros(2 * E, dtype=torch.int32)[::2])),
    ("y", dict(y=torch.zeros((TD, H)))), ("y", dict(ydt=moe.MOE_F32)), ("y", dict(y=torch.zeros((TD, H), dtype=torch.float16))),
    ("y", dict(y=torch.zeros((TD - 1, H), dtype=BF16))), ("y", dict(y=torch.zeros((TD, H + 8), dtype=BF16)[:, :H])),
    ("slot_pool", dict(pool=torch.zeros((1, 6000 * 2), dtype=U8))), ("slot_pool", dict(pool=torch.zeros((E, 40000), dtype=U8)[:, ::2])),
    ("shared_w", dict(shared=torch.zeros(12287, dtype=U8), ish=32)), ("shared_w", dict(shared=torch.zeros(24576, dtype=U8)[::2], ish=32)),
    ("workspace", dict(ws=torch.zeros(1, dtype=U8).expand(1 << 20)))])
def test_layer(what, change):
    _refused(what, lambda: _layer(**change))


def _pack(fmt, **change):
    group = 32 if fmt == moe.MOE_MXFP4 else 64
    a = dict(codes=torch.zeros((N, K // 2), dtype=U8), zeros=None,
             scales=torch.zeros((N, K // group), dtype=U8 if fmt == moe.MOE_MXFP4 else torch.float16),
             w=torch.zeros(moe.moe_w4_bytes(fmt, N, K, group), dtype=U8))
    a.update(change)
    moe.moe_w4_pack(fmt, a["codes"], a["scales"], a["zeros"], N, K, group, a["w"])


@pytest.mark.parametrize("fmt,what,change", [
    (moe.MOE_INT4, "codes", dict(codes=torch.zeros((N, K // 2), dtype=torch.int8))),
    (moe.MOE_INT4, "codes", dict(codes=torch.zeros((N, K), dtype=U8))),           # one code a byte
    (moe.MOE_INT4, "codes", dict(codes=torch.zeros((N - 1, K // 2), dtype=U8))),
    (moe.MOE_INT4, "codes", dict(codes=torch.zeros((N + 1, K // 2), dtype=U8))),
    (moe.MOE_INT4, "codes", dict(codes=torch.zeros((N, K), dtype=U8)[:, ::2])),
    (moe.MOE_MXFP4, "codes", dict(codes=torch.zeros((K // 2, N + 8), dtype=U8).t()[:N])),
    (moe.MOE_INT4, "codes", dict(codes=torch.zeros((N, K // 8), dtype=torch.int32))),
    (moe.MOE_INT4, "scales", dict(scales=torch.zeros((N, 1), dtype=BF16))),
    (moe.MOE_INT4, "scales", dict(scales=torch.zeros((N, 1)))),
    (moe.MOE_INT4, "scales", dict(scales=torch.zeros((1, N), dtype=torch.float16))),
    (moe.MOE_INT4, "scales", dict(scales=torch.zeros((N, 2), dtype=torch.float16))),
    (moe.MOE_MXFP4, "scales", dict(scales=torch.zeros((N, 2), dtype=torch.float16))),
    (moe.MOE_MXFP4, "scales", dict(scales=torch.zeros((N, 1), dtype=U8))),
    (moe.MOE_INT4, "zeros", dict(zeros=torch.zeros((N, 1), dtype=torch.int8))),
    (moe.MOE_INT4, "zeros", dict(zeros=torch.zeros((N, 1), dtype=torch.float16))),
    (moe.MOE_INT4, "zeros", dict(zeros=torch.zeros((N // 2, 1), dtype=U8))),
    (moe.MOE_INT4, "zeros", dict(zeros=torch.zeros((N, 2), dtype=U8)[:, :1])),
    (moe.MOE_INT4, "w", dict(w=torch.zeros(1, dtype=U8).expand(1 << 20)))])
def test_pack(fmt, what, change):
    _refused(what, lambda: _pack(fmt, **change))


def test_types_that_pass():
    """The types of the same bits go on to the look at the device, which refuses CPU tensors or has none."""
    for fmt, change in ((moe.MOE_MXFP4, {}), (moe.MOE_INT4, {}),
                        (moe.MOE_MXFP4, dict(scales=torch.zeros((N, 2), dtype=U8).view(torch.float8_e8m0fnu))),
                        (moe.MOE_MXFP4, dict(codes=torch.zeros((N, K // 2), dtype=U8).view(torch.float4_e2m1fn_x2))),
                        (moe.MOE_INT4, dict(scales=torch.zeros((N, 1), dtype=torch.int16))),
                        (moe.MOE_INT4, dict(codes=torch.zeros(N * K // 2, dtype=U8)))):
        with pytest.raises((moe.MoeError, RuntimeError)) as e:
            _pack(fmt, **change)
        assert not isinstance(e.value, moe.MoeError) or "device" in str(e.value)
