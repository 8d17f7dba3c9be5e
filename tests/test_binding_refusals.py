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
