"""Cases of the few-token operators: the whole MoE layer (routing, experts and the
weighted sum in one call) and the linear product with 4-bit weights.

``run`` computes either operator in elementary torch operations (``own`` false) or
through the library (``own`` true), from the same state.  Sizes are those of the
layer workloads (hidden 2048, intermediate 512, 256 + 1 experts, top-8 in bf16;
hidden 4096, intermediate 2048, 256 experts, top-6 in MXFP4), the projections of
such a layer, and odd ones.
"""
import math

import torch

own = False

BF16, MXFP4, INT4 = 1, 2, 4  # the library's weight type codes

# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def _layer(name, wdt, T, H, I, E, k, shared, skew):
    c = dict(op="layer", wdt=wdt, T=T, H=H, I=I, E=E, k=k, shared=shared, skew=skew)
    return dict(c, name=name) if name else c


def _linear(name, wdt, T, N, K, group, bias, f32_out):
    c = dict(op="linear", wdt=wdt, T=T, N=N, K=K, group=group, bias=bias, f32_out=f32_out)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one stream of text, one token at a time: what a single user waits for
        _layer("layer_bf16_t1", BF16, 1, 2048, 512, 256, 8, 512, 0.0),
        # a handful of streams, or a short draft being verified
        _layer("layer_bf16_t4", BF16, 4, 2048, 512, 256, 8, 512, 0.0),
        # a small serving batch: about a hundred different experts
        _layer("layer_bf16_t16", BF16, 16, 2048, 512, 256, 8, 512, 0.0),
        # the large 4-bit layer for one token, a small and a full decode batch, with
        # experts of skewed popularity
        _layer("layer_mxfp4_t1", MXFP4, 1, 4096, 2048, 256, 6, 0, 1.1),
        _layer("layer_mxfp4_t8", MXFP4, 8, 4096, 2048, 256, 6, 0, 1.1),
        _layer("layer_mxfp4_t64", MXFP4, 64, 4096, 2048, 256, 6, 0, 1.1),
        # a projection of one token: hidden to hidden
        _linear("linear_int4_t1", INT4, 1, 2048, 2048, 128, False, False),
        # fused projections of one token in the MXFP4 layer's width
        _linear("linear_mxfp4_t1", MXFP4, 1, 8192, 4096, 32, False, False),
        # fine groups, few tokens, a bias
        _linear("linear_int4_g32_t4", INT4, 4, 8192, 4096, 32, True, False),
        # ragged everywhere: rows past the last tile, a partial last group, odd tokens
        _linear("linear_int4_g64_odd", INT4, 7, 1003, 2080, 64, True, True),
        # the head over a vocabulary, logits in f32: a small and a full batch
        _linear("linear_mxfp4_head_t16", MXFP4, 16, 65536, 4096, 32, False, True),
        _linear("linear_int4_head_t64", INT4, 64, 65536, 4096, 128, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    cap = max(work(c)["bytes"] for c in listed())
    while True:
        if rng.random() < 0.5:
            wdt = rng.choice([BF16, MXFP4])
            H, I = 32 * _log(rng, 8, 128), 32 * _log(rng, 2, 64)
            E = _log(rng, 8, 256)
            k = rng.randint(1, 8)
            T = _log(rng, 1, 64)
            shared = rng.choice([0, 0, I, 32 * _log(rng, 2, 32)])
            if E * _expert_bytes(wdt, H, I) > 4 << 30:
                continue
            c = _layer(None, wdt, T, H, I, E, k, shared, rng.choice([0.0, 1.1]))
        else:
            wdt = rng.choice([MXFP4, INT4, INT4])
            group = 32 if wdt == MXFP4 else rng.choice([32, 64, 128])
            c = _linear(None, wdt, _log(rng, 1, 64), _log(rng, 100, 65536), 32 * _log(rng, 8, 256), group,
                        rng.random() < 0.3, rng.random() < 0.5)
        if work(c)["bytes"] <= cap:
            return c


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------


def _active(c):
    """Mean number of distinct experts a batch of this case routes to (16 draws)."""
    g = torch.Generator().manual_seed(7)
    n = 0
    for _ in range(16):
        z = torch.randn((c["T"], c["E"]), generator=g) - c["skew"] * torch.log1p(torch.arange(c["E"]).float())
        n += len(torch.unique(z.topk(c["k"]).indices))
    return n / 16


def work(case):
    c = case
    if c["op"] == "layer":
        T, H, k = c["T"], c["H"], c["k"]
        per = 3 * H * (2 if c["wdt"] == BF16 else 17 / 32)  # bytes per intermediate column of an expert
        weights = (_active(c) * c["I"] + c["shared"]) * per
        io = T * H * 2 * 2 + T * c["E"] * 4 + T * k * 8  # x, y, logits, ids and gate weights
        return {"bytes": weights + io, "flops": 2.0 * 3 * H * T * (k * c["I"] + c["shared"])}
    T, N, K = c["T"], c["N"], c["K"]
    groups = -(-K // c["group"])
    io = T * K * 2 + T * N * (4 if c["f32_out"] else 2) + (4 * N if c["bias"] else 0)
    return {"bytes": N * K / 2 + N * groups * (1 if c["wdt"] == MXFP4 else 3) + io, "flops": 2.0 * T * N * K}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _slot_parts(wdt, H, I):
    """(first byte, rows, columns, steps of columns) of W13 and W2 in an expert slot, the
    first bytes of their scale blocks (MXFP4), and the slot's size."""
    ks = 32 if wdt == BF16 else 128
    n13, n2 = -(-H // ks), -(-I // ks)
    b13, b2 = 2 * I // 16 * n13 * 1024, H // 16 * n2 * 1024
    if wdt == BF16:
        return (0, 2 * I, H, n13), (b13, H, I, n2), None, None, b13 + b2
    s13 = 2 * I // 16 * (-(-n13 // 16)) * 1024
    s2 = H // 16 * (-(-n2 // 16)) * 1024
    return (0, 2 * I, H, n13), (b13, H, I, n2), b13 + b2, b13 + b2 + s13, b13 + b2 + s13 + s2


def _expert_bytes(wdt, H, I):
    return _slot_parts(wdt, H, I)[4]


def _random_e2m1_bytes(shape, g, dev):
    """Bytes of two E2M1 codes each, of normal draws (standard deviation 2.56 steps: 0.02
    under a scale of 2^-7), drawn through a table of the format's nearest codes."""
    mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=dev)
    q = (torch.arange(256, device=dev, dtype=torch.float32) + 0.5) / 256
    v = torch.erfinv(2 * q - 1) * math.sqrt(2) * 2.56
    code = (v.abs()[:, None] - mags[None, :]).abs().argmin(1).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    lo = torch.randint(0, 256, shape, dtype=torch.uint8, device=dev, generator=g)
    hi = torch.randint(0, 256, shape, dtype=torch.uint8, device=dev, generator=g)
    return code[lo.int()] | (code[hi.int()] << 4)


def _random_slots(wdt, n, H, I, g, dev):
    """n experts with weights of standard deviation about 0.02, in the slot layout.  Every
    element is an independent draw, so only the padding has to be placed."""
    m13, m2, s13, s2, nb = _slot_parts(wdt, H, I)
    out = torch.zeros((n, nb), dtype=torch.uint8, device=dev)
    step = max(1, (256 << 20) // nb)
    for e in range(0, n, step):
        m = min(n, e + step) - e
        if wdt == BF16:
            w = torch.randn((m, nb // 2), generator=g, device=dev) * 0.02
            out[e:e + m] = w.to(torch.bfloat16).view(torch.uint8)
            continue
        for (at, rows, K, nk), sat in ((m13, s13), (m2, s2)):
            rt, nb16 = rows // 16, -(-nk // 16)
            codes = _random_e2m1_bytes((m, rt, nk, 4, 16, 16), g, dev)
            live = (torch.arange(nk * 4, device=dev) < K // 32).view(nk, 4)
            codes *= live[None, None, :, :, None, None]
            out[e:e + m, at:at + rt * nk * 1024] = codes.reshape(m, -1)
            sc = torch.randint(119, 122, (m, rt, nb16 * 16, 4, 16), dtype=torch.uint8, device=dev, generator=g)
            pad = (torch.arange(nb16 * 64, device=dev) < K // 32).view(nb16 * 16, 4)
            sc *= pad[None, None, :, :, None]
            # in a block of 16 steps, lane (group, row) owns 16 consecutive bytes
            sc = sc.view(m, rt, nb16, 16, 4, 16).permute(0, 1, 2, 4, 5, 3)
            out[e:e + m, sat:sat + rt * nb16 * 1024] = sc.reshape(m, -1)
    return out


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 12345)
    s = dict(case=c)
    if c["op"] == "layer":
        T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
        s["pool"] = _random_slots(c["wdt"], E, H, I, g, dev)
        s["shared"] = _random_slots(c["wdt"], 1, H, c["shared"], g, dev)[0] if c["shared"] else None
        s["slots"] = torch.randperm(E, generator=g, device=dev).to(torch.int32)
        s["x"] = torch.randn((T, H), generator=g, device=dev).to(torch.bfloat16)
        rank = torch.randperm(E, generator=g, device=dev).float()
        s["logits"] = torch.randn((T, E), generator=g, device=dev) - c["skew"] * torch.log1p(rank)
        if own:
            from routed_expert_ffn_layer_amd import layer
            s["buffers"] = layer.LayerBuffers(T, E, k, H, I, c["wdt"], I_shared=c["shared"])
        return s
    T, N, K = c["T"], c["N"], c["K"]
    groups = -(-K // c["group"])
    s["x"] = torch.randn((T, K), generator=g, device=dev).to(torch.bfloat16)
    s["bias"] = torch.randn((N,), generator=g, device=dev) if c["bias"] else None
    if c["wdt"] == MXFP4:
        s["codes"] = _random_e2m1_bytes((N, K // 2), g, dev)
        s["scales"] = torch.randint(119, 122, (N, groups), dtype=torch.uint8, device=dev, generator=g)
        s["zeros"] = None
    else:
        s["codes"] = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=dev, generator=g)
        s["scales"] = ((0.5 + torch.rand((N, groups), generator=g, device=dev)) * 0.005).to(torch.float16)
        s["zeros"] = torch.randint(5, 11, (N, groups), dtype=torch.uint8, device=dev, generator=g)
    if own:
        from routed_expert_ffn_layer_amd import moe
        w = torch.empty(moe.moe_w4_bytes(c["wdt"], N, K, c["group"]), dtype=torch.uint8, device=dev)
        moe.moe_w4_pack(c["wdt"], s["codes"], s["scales"], s["zeros"], N, K, c["group"], w)
        s["w"] = w
        s["y"] = torch.empty((T, N), dtype=torch.float32 if c["f32_out"] else torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    c = s["case"]
    if c["op"] == "layer":
        from routed_expert_ffn_layer_amd import layer
        b = s["buffers"]
        y = layer.forward_decode(b, s["logits"], s["x"], s["pool"], s["pool"].shape[1], s["slots"], s["shared"])
        return y, b.topk_ids, b.topk_w
    from routed_expert_ffn_layer_amd import moe
    moe.moe_w4_linear(c["wdt"], s["w"], c["N"], c["K"], c["group"], s["x"], s["bias"], s["y"])
    return s["y"]


def _e2m1(codes):
    """E2M1 codes (integers 0..15) to their values in f32."""
    mag = codes & 7
    exp, man = mag >> 1, (mag & 1).float()
    v = torch.where(exp == 0, man * 0.5, (1 + 0.5 * man) * torch.exp2(exp.float() - 1))
    return torch.where(codes >= 8, -v, v)


def _nibbles(b):
    """Bytes [..., n] to codes [..., 2n], the low nibble first."""
    return torch.stack((b & 15, b >> 4), dim=-1).flatten(-2)


def _matrix(slot, wdt, part, sat):
    """A tiled matrix of a slot as f32 [rows][K]."""
    at, rows, K, nk = part
    rt = rows // 16
    b = slot[at:at + rt * nk * 1024]
    if wdt == BF16:
        w = b.view(torch.bfloat16).view(rt, nk, 4, 16, 8).float()
        return w.permute(0, 3, 1, 2, 4).reshape(rows, K)
    w = _e2m1(_nibbles(b.view(rt, nk, 4, 16, 16)))
    nb16 = -(-nk // 16)
    sc = slot[sat:sat + rt * nb16 * 1024].view(rt, nb16, 4, 16, 16)
    sc = torch.exp2(sc.float() - 127).permute(0, 1, 4, 2, 3).reshape(rt, nb16 * 16, 4, 16)[:, :nk]
    return (w * sc[..., None]).permute(0, 3, 1, 2, 4).reshape(rows, nk * 128)[:, :K]


def _expert(slot, wdt, x, H, I):
    """SwiGLU expert of one slot on the rows x [n][H] f32."""
    m13, m2, s13, s2, _ = _slot_parts(wdt, H, I)
    gu = x @ _matrix(slot, wdt, m13, s13).t()
    gu = gu.view(-1, I // 8, 2, 8)  # tiles of 8 gate rows and the 8 up rows beside them
    gate, up = gu[:, :, 0].reshape(-1, I), gu[:, :, 1].reshape(-1, I)
    return (gate * torch.sigmoid(gate) * up) @ _matrix(slot, wdt, m2, s2).t()


def _run_plain(s):
    c = s["case"]
    x = s["x"].float()
    if c["op"] == "layer":
        H, I, k = c["H"], c["I"], c["k"]
        vals, ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)
        vals, ids = vals[:, :k], ids[:, :k]
        ex = torch.exp(vals - vals[:, :1])
        w = ex / ex.sum(1, keepdim=True)
        y = torch.zeros((c["T"], H), device=x.device)
        slots = s["slots"][ids].long()
        for t in range(c["T"]):
            for j in range(k):
                slot = s["pool"].index_select(0, slots[t, j:j + 1])[0]
                y[t] += w[t, j] * _expert(slot, c["wdt"], x[t:t + 1], H, I)[0]
        if c["shared"]:
            y += _expert(s["shared"], c["wdt"], x, H, c["shared"])
        return y.to(torch.bfloat16), ids.to(torch.int32), w
    K = c["K"]
    q = _nibbles(s["codes"])
    per = s["scales"].float() if c["wdt"] == INT4 else torch.exp2(s["scales"].float() - 127)
    per = per.repeat_interleave(c["group"], 1)[:, :K]
    if c["wdt"] == MXFP4:
        w = _e2m1(q) * per
    else:
        w = (q.float() - s["zeros"].float().repeat_interleave(c["group"], 1)[:, :K]) * per
    y = x @ w.t()
    if s["bias"] is not None:
        y += s["bias"]
    return y if c["f32_out"] else y.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

_E2M1_TABLE = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _element_table(dev):
    return torch.tensor(_E2M1_TABLE, dtype=torch.float64, device=dev)


def _exact_rows(slot, wdt, part, sat):
    """Rows of a tiled matrix gathered element by element from the layout's definition."""
    at, rows, K, nk = part
    r = torch.arange(rows, device=slot.device)[:, None]
    k = torch.arange(K, device=slot.device)[None, :]
    if wdt == BF16:
        tile = (r // 16) * nk + k // 32
        idx = at // 2 + tile * 512 + (16 * (k % 32 // 8) + r % 16) * 8 + k % 8
        return slot.view(torch.bfloat16)[idx].double()
    step, frag = k // 128, 16 * (k % 128 // 32) + r % 16
    byte = slot[at + ((r // 16) * nk + step) * 1024 + frag * 16 + k % 32 // 2].int()
    code = torch.where(k % 2 == 1, byte >> 4, byte & 15)
    sc = slot[sat + ((r // 16) * (-(-nk // 16)) + step // 16) * 1024 + frag * 16 + step % 16].double()
    return _element_table(slot.device)[code] * torch.pow(2.0, sc - 127)


def _exact_expert(slot, wdt, x, H, I):
    m13, m2, s13, s2, _ = _slot_parts(wdt, H, I)
    w13 = _exact_rows(slot, wdt, m13, s13)
    i = torch.arange(I, device=slot.device)
    gate = x @ w13[16 * (i // 8) + i % 8].t()
    up = x @ w13[16 * (i // 8) + 8 + i % 8].t()
    return (gate / (1 + torch.exp(-gate)) * up) @ _exact_rows(slot, wdt, m2, s2).t()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    x = s["x"].double()
    if c["op"] == "layer":
        T, k, E = c["T"], c["k"], c["E"]
        rows = s["logits"].double().tolist()
        ids = torch.tensor([sorted(range(E), key=lambda e: (-row[e], e))[:k] for row in rows], device=x.device)
        w = torch.softmax(torch.gather(s["logits"].double(), 1, ids), 1)
        y = torch.zeros((T, c["H"]), dtype=torch.float64, device=x.device)
        for e in torch.unique(ids).tolist():
            t, j = torch.nonzero(ids == e, as_tuple=True)
            out = _exact_expert(s["pool"][int(s["slots"][e])], c["wdt"], x[t], c["H"], c["I"])
            y.index_add_(0, t, out * w[t, j][:, None])
        if c["shared"]:
            y += _exact_expert(s["shared"], c["wdt"], x, c["H"], c["shared"])
        return y, ids.to(torch.int32), w
    N, K, G = c["N"], c["K"], c["group"]
    k = torch.arange(K, device=x.device)
    y = torch.empty((c["T"], N), dtype=torch.float64, device=x.device)
    for n in range(0, N, 8192):
        byte = s["codes"][n:n + 8192][:, k // 2].int()
        code = torch.where(k % 2 == 1, byte >> 4, byte & 15)
        sc = s["scales"][n:n + 8192].double()[:, k // G]
        if c["wdt"] == MXFP4:
            w = _element_table(x.device)[code] * torch.pow(2.0, sc - 127)
        else:
            w = (code - s["zeros"][n:n + 8192].int()[:, k // G]) * sc
        y[:, n:n + 8192] = x @ w.t()
    return y + s["bias"].double() if s["bias"] is not None else y
