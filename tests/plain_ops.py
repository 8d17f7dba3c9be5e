"""Plain 64-bit forms of the operators around the experts, and the bounds of their tests.

Bounds count roundings: u = 2^-24 is half a step of f32, relative, and a result stored as bf16 is off
by another half step, 2^-8."""
import math

import torch

U = 2.0 ** -24
RMS, LAYER = 1, 2
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2 if dtype is torch.bfloat16 else U


def stored(ref, tol, dtype):
    """Bound of a result that is within tol of ref before it is rounded to dtype (the subnormals of either
    type start at 2^-126: half a step there is 2^-134 in bf16 and less in f32)."""
    return tol + (ref.abs() + tol) * half_step(dtype) + 2.0 ** -134


def check(got, ref, tol, what=""):
    """got within tol of ref, element by element; infinities and NaN where ref has them."""
    got, ref = got.detach().double().cpu(), ref.double().cpu()
    tol = torch.as_tensor(tol, dtype=torch.float64).cpu().expand_as(ref)
    fine = torch.isfinite(ref)
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} for {tuple(ref.shape)}"
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    rest = ~fine & ~torch.isnan(ref)
    assert torch.equal(got[rest], ref[rest]), f"{what}: other infinities"
    bad = fine & ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i].item()!r} for "
                             f"{ref[i].item()!r}, bound {tol[i].item():.3g}")


def unit(v, kind, eps):
    """The norm without weights, and the divisor of each row."""
    d = v - v.mean(1, keepdim=True) if kind == LAYER else v
    dev = torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    return d / dev, d, dev


def norm(v, dv, kind, w, b, eps):
    """Norm of rows v (f64) that the library holds within dv: (result, bound).

    Sums of H terms by up to 32 in a lane, then 6 + 16 joins, on squares that carry 3 roundings: under
    64 u relative in the divisor's square, 32 u in the divisor, and a few for root, quotient and product:
    64 u of the result covers them; layer norm: d carries one rounding of its own, and the mean taken off
    d, itself a sum of H rounded terms in the same 32 + 22 additions, is off by up to 55 u mean|d| <= 64 u
    mean|d| whatever the element, which an element next to the mean has to bear in full.  An error dv of the
    row moves d by dv and its mean, and the divisor by at most |dv| / |d| in the 2-norm."""
    n, d, dev = unit(v, kind, eps)
    scale = w.double() if w is not None else torch.ones(v.shape[1], dtype=torch.float64)
    shift = (dv * dv).sum(1, keepdim=True).sqrt() / (d * d).sum(1, keepdim=True).sqrt().clamp(min=1e-300)
    tol = (n * scale).abs() * (64 * U + shift) + scale.abs() * dv / dev
    if kind == LAYER:
        tol = tol + scale.abs() * (dv.mean(1, keepdim=True) + 64 * U * d.abs().mean(1, keepdim=True)) / dev
    out = n * scale + (b.double() if b is not None else 0)
    if b is not None:
        tol = tol + 2 * U * out.abs()
    return out, tol


def block_norm(block, post, gate, bs, res, rs, pre, eps):
    """((r', bound), (x, bound) or None), before rounding to the stored types; norms as (kind, w, b) or None."""
    zero = lambda v: torch.zeros_like(v)  # noqa: E731
    bs, rs = float(torch.tensor(bs)), float(torch.tensor(rs))  # f32 arguments
    eps = float(torch.tensor(eps))
    if block is not None:
        n, tol = block.double(), zero(block.double())
        if post:
            n, tol = norm(n, tol, *post, eps)
        if gate is not None:
            n, tol = n * gate.double(), (tol + U * n.abs()) * gate.double().abs()
        r, tol = bs * n, abs(bs) * tol + 2 * U * (bs * n).abs()
        if res is not None:
            r, tol = r + rs * res.double(), tol + 2 * U * (rs * res.double()).abs()
        tol = tol + 2 * U * r.abs()
    else:
        r = rs * res.double()
        tol = U * r.abs()
    return (r, tol), (norm(r, tol, *pre, eps) if pre else (r, tol))


def act(v, name):
    if name == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * torch.erfc(-v / math.sqrt(2)) / 2
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def act_bound(v, tol, name):
    """Bound of act(v + error up to tol): slopes stay below 1.13; the exponentials take arguments with
    one or (GELU) four roundings, which makes a relative error of the argument times that.  The reciprocal
    1 / (1 + e^z) has no subnormal results: past e^z = 2^126 it is 0, off by up to 2^-126, times |v|."""
    a = v.abs()
    tol = tol + a * 2.0 ** -126
    if name == "silu":
        own = act(v, name).abs() * (2 * a + 16) * U
    elif name == "gelu":  # erf within 1.5e-7; the tail q = erfc / 2 relative to its own size
        own = a * (0.75e-7 + torch.erfc(a / math.sqrt(2)) / 2 * (4 * a * a + 32) * U + 4 * U)
    elif name == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
        own = act(v, name).abs() * (16 * u + 16) * U
    else:
        return tol
    return 1.13 * tol + own


def linear(x, w, bias, name, res):
    """(y, bound) before the rounding to the stored type: K products added in any order, each addition
    off by one whole step at most (2 u: the matrix instruction may cut instead of round)."""
    x, w = x.double(), w.double()
    v, tol = x @ w.t(), (x.abs() @ w.abs().t()) * (2 * U * x.shape[1])
    if bias is not None:
        v = v + bias.double()
        tol = tol + U * v.abs()
    y, tol = act(v, name), act_bound(v, tol, name)
    if res is not None:
        y = y + res.double()
        tol = tol + 2 * U * y.abs()
    return y, tol


def order(ids, E):
    """counts, offsets, sorted_rows, inv_rows by the definition."""
    flat = ids.reshape(-1).tolist()
    of = [[] for _ in range(E)]
    for r, e in enumerate(flat):
        if 0 <= e < E:
            of[e].append(r)
    counts = [len(v) for v in of]
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    rows = [r for v in of for r in v]
    inv = [-1] * len(flat)
    for p, r in enumerate(rows):
        inv[r] = p
    return tuple(torch.tensor(v, dtype=torch.int32) for v in (counts, offsets, rows + [-1] * (len(flat) - len(rows)), inv))


def combine(rows, w, inv, T, n_rows):
    """(y, sum of magnitudes)."""
    k = inv.numel() // T
    at = inv.long().view(T, k)
    live = (at >= 0) & (at < n_rows)
    got = rows.double()[at.clamp(0, max(n_rows - 1, 0))] if n_rows else torch.zeros((T, k, rows.shape[1]), dtype=torch.float64)
    v = torch.where(live[..., None], w.double()[..., None] * got, torch.zeros((), dtype=torch.float64))
    return v.sum(1), v.abs().sum(1)
