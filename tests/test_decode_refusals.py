"""Calls of moe_layer_decode, moe_w4_pack and moe_w4_linear that are refused before any
device work, and the sizes they report (runs without a GPU)."""
import ctypes

import pytest

from routed_expert_ffn_layer_amd import moe

P = ctypes.c_void_p(1 << 20)
BAD = ctypes.c_void_p((1 << 20) + 8)  # not 16-byte aligned
EB = 2 * 3 * 64 * 32


def _layer(**kw):
    a = dict(wdt=moe.MOE_BF16, pool=P, stride=EB, slots=P, shared=None, ish=0, x=P, logits=P, T=4, k=2, E=8, H=64, I=32,
             ids=P, w=P, y=P, ydt=moe.MOE_BF16, ws=P, nws=1 << 20)
    a.update(kw)
    return moe.lib().moe_layer_decode(a["wdt"], a["pool"], a["stride"], a["slots"], a["shared"], a["ish"], a["x"],
                                      a["logits"], a["T"], a["k"], a["E"], a["H"], a["I"], a["ids"], a["w"], a["y"],
                                      a["ydt"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(wdt=9), moe.MOE_EINVAL), (dict(wdt=-1), moe.MOE_EINVAL), (dict(wdt=moe.MOE_INT4), moe.MOE_EINVAL),
    (dict(wdt=moe.MOE_F32, stride=1 << 20), moe.MOE_EUNSUPPORTED), (dict(wdt=moe.MOE_MXFP4_A8), moe.MOE_EUNSUPPORTED),
    (dict(T=-1), moe.MOE_EINVAL), (dict(k=0), moe.MOE_EINVAL), (dict(k=9), moe.MOE_EINVAL), (dict(E=0), moe.MOE_EINVAL),
    (dict(E=1025), moe.MOE_EINVAL), (dict(H=48), moe.MOE_EINVAL), (dict(I=16), moe.MOE_EINVAL), (dict(H=0), moe.MOE_EINVAL),
    (dict(T=65, k=1), moe.MOE_EUNSUPPORTED), (dict(T=64, k=9, E=16), moe.MOE_EUNSUPPORTED),
    (dict(ydt=2), moe.MOE_EINVAL), (dict(stride=EB - 16), moe.MOE_EINVAL), (dict(stride=EB + 8), moe.MOE_EINVAL),
    (dict(shared=P, ish=16), moe.MOE_EINVAL), (dict(shared=P, ish=0), moe.MOE_EINVAL), (dict(shared=BAD, ish=32), moe.MOE_EINVAL),
    (dict(nws=4 * 2 * 32 * 4 + 13327), moe.MOE_ECAPACITY),
    (dict(shared=P, ish=64, nws=12 * 64 * 4 + 13327), moe.MOE_ECAPACITY),
    (dict(H=65568, stride=1 << 24), moe.MOE_EUNSUPPORTED),
    (dict(T=64, k=8, H=32, I=1 << 20, stride=1 << 30, nws=1 << 40), moe.MOE_EUNSUPPORTED),  # 512 rows of 4 MiB
    (dict(wdt=moe.MOE_BF16, H=32768, I=16384, stride=1 << 40, nws=1 << 30), moe.MOE_EUNSUPPORTED),  # experts of 3 GiB
] + [({n: v}, moe.MOE_EINVAL) for n in ("pool", "slots", "x", "ids", "w", "y", "ws") for v in (None, BAD)]
  + [(dict(logits=BAD), moe.MOE_EINVAL)])
def test_layer_refusals(kw, status):
    assert _layer(**kw) == status
    assert moe.lib().moe_last_error()


def test_layer_without_tokens_needs_no_buffers():
    assert _layer(T=0, pool=None, slots=None, x=None, logits=None, ids=None, w=None, y=None, ws=None, nws=0) == moe.MOE_OK


def test_layer_workspace():
    ws = moe.moe_layer_decode_workspace
    # two bf16 per element of the intermediate, in whole 256 bytes, then the routing: 16 bytes, 16 per run, two integers per pair
    plan = 16 + 16 * (moe.MOE_LAYER_DECODE_MAX_PAIRS + 64) + 2 * 4 * moe.MOE_LAYER_DECODE_MAX_PAIRS
    assert ws(4, 2, 8, 64, 32, 0, moe.MOE_BF16) == 4 * 2 * 32 * 4 + plan
    assert ws(4, 2, 8, 64, 32, 64, moe.MOE_BF16) == (8 + 4) * 64 * 4 + plan
    assert ws(4, 2, 8, 64, 32, 64, moe.MOE_MXFP4) == (8 + 4) * 128 * 4 + plan  # rows of whole 128 columns
    assert ws(1, 1, 8, 64, 32, 0, moe.MOE_BF16) == 256 + plan
    assert ws(4, 2, 8, 64, 32, 0, moe.MOE_F32) == 0 and ws(-1, 2, 8, 64, 32, 0, moe.MOE_BF16) == 0


def _linear(**kw):
    a = dict(fmt=moe.MOE_INT4, w=P, N=40, K=256, group=64, x=P, x_ld=256, T=3, bias=None, y=P, y_ld=40, ydt=moe.MOE_F32)
    a.update(kw)
    return moe.lib().moe_w4_linear(a["fmt"], a["w"], a["N"], a["K"], a["group"], a["x"], a["x_ld"], a["T"], a["bias"],
                                   a["y"], a["y_ld"], a["ydt"], None)


SHAPES = [dict(fmt=1), dict(fmt=3), dict(N=0), dict(N=-5), dict(N=(1 << 30) + 1, K=32, x_ld=32, y_ld=1 << 31), dict(K=0), dict(K=48), dict(K=-32), dict(K=(1 << 20) + 32, x_ld=1 << 22),
          dict(group=16), dict(group=256), dict(group=0), dict(fmt=moe.MOE_MXFP4, group=64),
          dict(N=1 << 30, K=1 << 20, x_ld=1 << 20, y_ld=1 << 30)]


@pytest.mark.parametrize("kw", SHAPES + [
    dict(T=-1), dict(T=(1 << 19) + 1), dict(ydt=2), dict(ydt=-1), dict(x_ld=248), dict(x_ld=260), dict(x_ld=(1 << 22) + 8),
    dict(y_ld=39), dict(w=None), dict(w=BAD), dict(x=None), dict(x=BAD), dict(y=None), dict(y=BAD), dict(bias=BAD)])
def test_linear_refusals(kw):
    assert _linear(**kw) == moe.MOE_EINVAL


def test_linear_without_tokens_needs_no_buffers():
    assert _linear(T=0, w=None, x=None, y=None) == moe.MOE_OK


@pytest.mark.parametrize("kw", SHAPES + [dict(codes=None), dict(codes=BAD), dict(scales=None), dict(scales=BAD), dict(w=None),
                                         dict(w=BAD), dict(fmt=moe.MOE_MXFP4, group=32, zeros=P)])
def test_pack_refusals(kw):
    a = dict(fmt=moe.MOE_INT4, codes=P, scales=P, zeros=None, N=40, K=256, group=64, w=P)
    a.update({k: v for k, v in kw.items() if not k.endswith("_ld")})
    assert moe.lib().moe_w4_pack(a["fmt"], a["codes"], a["scales"], a["zeros"], a["N"], a["K"], a["group"], a["w"],
                                 None) == moe.MOE_EINVAL


def test_packed_bytes():
    b = moe.moe_w4_bytes
    assert b(moe.MOE_MXFP4, 4096, 4096, 32) == 4096 * 2048 + 256 * 2 * 1024
    assert b(moe.MOE_INT4, 40, 256, 64) == 3 * 2 * 1024 + 3 * 256
    assert b(moe.MOE_INT4, 16, 2080, 128) == 17 * 1024 + 5 * 256  # 17 groups: 5 blocks of 4
    assert b(moe.MOE_INT4, 16, 100, 128) == 0 and b(7, 16, 128, 128) == 0
