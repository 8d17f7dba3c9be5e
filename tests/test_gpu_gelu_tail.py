"""GELU of moe_linear over its whole range, the tail to its own digits.

Bound (u = 2^-24): P(Z > a) carries 3 roundings of its exponent a^2 / 2 (the square, the constant, their product), that
is 1.5 a^2 u, and 24 u for the reciprocal (4 u of its argument and itself, which t P(t) takes up to 3 times), 8 steps of a
polynomial whose partial sums stay below the last, the fit, the exponential and two products.  z P(Z < z) is that times
|z| below 0, one rounding more; above 0 the tail is taken from 1, two.  The exponential has no subnormal results."""
import math

import pytest
import torch

import plain_ops as P
from routed_expert_ffn_layer_amd import moe

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _values(dt):
    v = torch.cat([torch.linspace(-14, 14, 4001), torch.tensor([0.0, 1e-20, -1e-20, -2.0 ** -130, 100.0, -100.0, 3e4, -3e4, -1e30, 3e38])])
    return torch.cat([v, torch.zeros(-len(v) % 8)]).to(dt)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("ydt", [F32, BF16])
@pytest.mark.parametrize("T,N", [(3, 8), (0, 8), (0, 520)])
def test_tail(dt, ydt, T, N):
    """T tokens at a time (0: all): every value passes to the activation as it is, through the three kernels."""
    v = _values(dt)
    x = torch.zeros((len(v), 8), dtype=dt)
    x[:, 2] = v
    w, x = torch.ones((N, 8), dtype=dt, device="cuda"), x.cuda()
    y = torch.empty((len(v), N), dtype=ydt, device="cuda")
    step = T if T else len(v)
    for lo in range(0, len(v), step):
        moe.moe_linear(w, x[lo:lo + step], None, moe.MOE_ACT_GELU, None, y[lo:lo + step])
    torch.cuda.synchronize()
    z = v.double()
    a = z.abs()
    q = torch.erfc(a / math.sqrt(2)) / 2
    ref = P.act(z, "gelu")
    tail = a * q * (1.5 * a * a + 24) * P.U
    tol = tail + torch.where(z < 0, ref.abs(), 2 * a) * P.U + a * 2.0 ** -126
    P.check(y, ref[:, None].expand(-1, N), P.stored(ref, tol, ydt)[:, None])
