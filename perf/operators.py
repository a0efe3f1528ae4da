"""Cases that time the mixture-of-experts operators and the 4-bit group products.

``own = False`` computes each operator in elementary torch operations; ``own = True`` calls the
package.  ``exact`` computes the same outputs in 64 bits from the definitions, apart from the plain form.

Operators:
  route    scores of E experts -> top-k ids and weights (softmax or sigmoid, balance bias, groups)
  matmul   y[t, s] = x[t] . W[ids[t, s]]^T, the experts' weights in GGUF blocks
  glu      h[t, s] = act(x[t] . Wg^T) * (x[t] . Wu^T), the experts' gate and up projections
  combine  y[t] = sum_s weights[t, s] (h[t, s] . W[ids[t, s]]^T), the experts' down projection
  w4       y = x . W^T, W in 4-bit codes with a scale (and zero point) per group of a row
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FMT_ID = {"Q4_0": 2, "Q5_0": 6, "Q8_0": 8, "Q4_K": 12, "Q6_K": 14}
BLOCK = {"Q4_0": (32, 18), "Q5_0": (32, 22), "Q8_0": (32, 34), "Q4_K": (256, 144), "Q6_K": (256, 210)}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one token of a served model choosing among 64 experts: launch latency
        dict(name="route_1x64", op="route", T=1, E=64, k=8, score="softmax", bias=False, groups=1, top_groups=1,
             group_top=1, renorm=True, scale=1.0, dtype="f32", masked=False),
        # a ragged batch, groups of experts, some rows padding (every expert masked)
        dict(name="route_333x160_groups", op="route", T=333, E=160, k=6, score="softmax", bias=False, groups=8,
             top_groups=3, group_top=1, renorm=False, scale=16.0, dtype="bf16", masked=True),
        # a long prompt through sigmoid scores with a balance bias
        dict(name="route_8192x256_bias", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32", masked=False),
        # one token, a projection of the scale-up shape: weight bandwidth
        dict(name="w4_1x14336x4096_g128", op="w4", M=1, N=14336, K=4096, G=128, zeros=False, sdtype="f16", dtype="bf16"),
        # a few tokens, small groups with zero points, an odd number of rows
        dict(name="w4_7x1537x1536_g32_zeros", op="w4", M=7, N=1537, K=1536, G=32, zeros=True, sdtype="f16", dtype="f32"),
        # a prompt of 512 tokens: matrix rate
        dict(name="w4_512x14336x4096_g128", op="w4", M=512, N=14336, K=4096, G=128, zeros=True, sdtype="f16", dtype="bf16"),
        # gate and up of eight experts for one token
        dict(name="glu_1_q4k_64x1024x2048", op="glu", fmt="Q4_K", T=1, E=64, k=8, N=1024, K=2048, act="silu", dtype="bf16",
             pad=False),
        # gate and up for a prompt of 2048 tokens, 256 rows per expert on average
        dict(name="glu_2048_q4k_64x1024x2048", op="glu", fmt="Q4_K", T=2048, E=64, k=8, N=1024, K=2048, act="silu",
             dtype="bf16", pad=False),
        # down of eight experts for one token, weighted sum
        dict(name="combine_1_q6k_64x2048x1024", op="combine", fmt="Q6_K", T=1, E=64, k=8, N=2048, K=1024, dtype="bf16",
             pad=False),
        # down for a prompt, padding rows behind it
        dict(name="combine_1500_q8_64x2048x1024", op="combine", fmt="Q8_0", T=1500, E=64, k=8, N=2048, K=1024, dtype="f16",
             pad=True),
        # a small serving batch through small experts, f32 activations
        dict(name="matmul_19_q8_32x1536x576", op="matmul", fmt="Q8_0", T=19, E=32, k=4, N=1536, K=576, dtype="f32", pad=True),
        # a short prompt, few wide experts
        dict(name="matmul_307_q5_8x1536x1536", op="matmul", fmt="Q5_0", T=307, E=8, k=2, N=1536, K=1536, dtype="f32",
             pad=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "w4", "w4", "glu", "combine", "matmul"])
    if op == "route":
        gsize = rng.randint(2, 32)
        groups = rng.choice([1, 1, 2, 4, 8])
        E = gsize * groups
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, gsize * top_groups))
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, group_top=rng.randint(1, 2),
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16", "f16"]),
                    masked=rng.random() < 0.3)
    if op == "w4":
        G = rng.choice([32, 64, 128])
        K = G * max(1, _log(rng, 256, 8192) // G)
        N = _log(rng, 64, 14336)
        M = _log(rng, 1, 1024)
        while M * N * K > 512 * 14336 * 4096:
            M = (M + 1) // 2
        return dict(op=op, M=M, N=N, K=K, G=G, zeros=rng.random() < 0.5, sdtype=rng.choice(["f16", "bf16", "f32"]),
                    dtype=rng.choice(["f32", "bf16", "f16"]))
    fmt = rng.choice(sorted(BLOCK))
    qk = BLOCK[fmt][0]
    E = _log(rng, 4, 128)
    k = rng.randint(1, min(8, E))
    K = qk * max(1, _log(rng, 256, 4096) // qk)
    N = _log(rng, 64, 4096)
    while E * N * K > 64 * 1024 * 2048:
        E = (E + 1) // 2
    k = min(k, E)
    T = _log(rng, 1, 2048)
    while T * k * N * K > 2048 * 8 * 1024 * 2048:
        T = (T + 1) // 2
    case = dict(op=op, fmt=fmt, T=T, E=E, k=k, N=N, K=K, dtype=rng.choice(["f32", "bf16", "f16"]), pad=rng.random() < 0.3)
    if op == "glu":
        case["act"] = rng.choice(["silu", "gelu"])
    return case


def _distinct(case):
    # experts that at least one of the tokens chooses, were the choices even
    E, k, T = case["E"], case["k"], case["T"]
    return E * (1.0 - (1.0 - k / E) ** T)


def work(case):
    op = case["op"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * size[case["dtype"]] + T * k * 8 + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
    e = size[case["dtype"]]
    if op == "w4":
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        w = N * K // 2 + N * (K // G) * (size[case["sdtype"]] + (1 if case["zeros"] else 0))
        return {"bytes": w + e * M * (K + N), "flops": 2 * M * N * K}
    T, k, N, K = case["T"], case["k"], case["N"], case["K"]
    qk, qb = BLOCK[case["fmt"]]
    mats = 2 if op == "glu" else 1
    w = int(_distinct(case) * N * (K // qk * qb)) * mats
    xin = T * k * K if op == "combine" else T * K
    yout = T * N if op == "combine" else T * k * N
    return {"bytes": w + e * (xin + yout) + T * k * (8 if op == "combine" else 4), "flops": 2 * T * k * N * K * mats}


# ----------------------------------------------------------------- inputs ---

def _codes(gen, shape, mean, sigma, lo, hi):
    return torch.randn(shape, generator=gen, device=DEV).mul_(sigma).add_(mean).round_().clamp_(lo, hi).to(torch.int16)


def _half_bytes(v):
    return v.to(torch.float16).unsqueeze(-1).view(torch.uint8)


def _blocks(gen, fmt, rows, K):
    """Rows of GGUF blocks as trained weights give them: bell-shaped codes, one scale per block."""
    qk, _ = BLOCK[fmt]
    nb = K // qk
    s = 0.02 * (0.6 + 0.8 * torch.rand((rows, nb), generator=gen, device=DEV))  # a block's spread
    if fmt == "Q8_0":
        q = _codes(gen, (rows, nb, 32), 0, 50, -127, 127).to(torch.int8).view(torch.uint8)
        parts = [_half_bytes(s / 50), q]
    elif fmt in ("Q4_0", "Q5_0"):
        top, sig = (15, 3.2) if fmt == "Q4_0" else (31, 6.4)
        q = _codes(gen, (rows, nb, 32), (top + 1) / 2, sig, 0, top)
        lo = q & 15
        qs = (lo[..., :16] | (lo[..., 16:] << 4)).to(torch.uint8)
        parts = [_half_bytes(s / sig)]
        if fmt == "Q5_0":
            bits = (q >> 4).view(rows, nb, 4, 8)
            sh = torch.arange(8, device=DEV, dtype=torch.int16)
            parts.append((bits << sh).sum(-1).to(torch.uint8))
        parts.append(qs)
    elif fmt == "Q4_K":
        q = _codes(gen, (rows, nb, 8, 32), 7.5, 3.4, 0, 15)
        sc = torch.randint(24, 64, (rows, nb, 8), generator=gen, device=DEV, dtype=torch.int16)
        mn = (sc + torch.randint(-4, 5, (rows, nb, 8), generator=gen, device=DEV, dtype=torch.int16)).clamp_(0, 63)
        d = s / (3.4 * 44)
        first = (sc[..., :4] | ((sc[..., 4:] >> 4) << 6))
        second = (mn[..., :4] | ((mn[..., 4:] >> 4) << 6))
        third = ((sc[..., 4:] & 15) | ((mn[..., 4:] & 15) << 4))
        pairs = q.view(rows, nb, 4, 2, 32)
        qs = (pairs[..., 0, :] | (pairs[..., 1, :] << 4)).reshape(rows, nb, 128)
        parts = [_half_bytes(d), _half_bytes(d * 7.5), torch.cat([first, second, third, qs], -1).to(torch.uint8)]
    else:  # Q6_K
        q = _codes(gen, (rows, nb, 2, 4, 32), 32, 12, 0, 63)
        sc = torch.randint(50, 128, (rows, nb, 16), generator=gen, device=DEV, dtype=torch.int16)
        sc = sc * (1 - 2 * torch.randint(0, 2, (rows, nb, 16), generator=gen, device=DEV, dtype=torch.int16))
        lo, hi = q & 15, q >> 4
        ql = torch.stack([lo[..., 0, :] | (lo[..., 2, :] << 4), lo[..., 1, :] | (lo[..., 3, :] << 4)], -2)
        qh = hi[..., 0, :] | (hi[..., 1, :] << 2) | (hi[..., 2, :] << 4) | (hi[..., 3, :] << 6)
        parts = [ql.reshape(rows, nb, 128).to(torch.uint8), qh.reshape(rows, nb, 64).to(torch.uint8),
                 sc.to(torch.int8).view(torch.uint8), _half_bytes(s / (12 * 90))]
    return torch.cat(parts, -1).reshape(rows, -1)


def _choices(gen, T, E, k, pad):
    """Distinct experts per token, some experts more wanted than others; padding rows choose none."""
    want = torch.randn((T, E), generator=gen, device=DEV) + 0.5 * torch.randn((1, E), generator=gen, device=DEV)
    top = torch.topk(want, k, dim=1)
    ids = top.indices.to(torch.int32)
    weights = torch.softmax(top.values, 1)
    if pad:
        last = max(1, T - max(1, T // 16))
        if last < T:
            ids[last:] = -1
            weights[last:] = 0
    return ids.contiguous(), weights.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": case, "op": op}
    if op == "route":
        T, E = case["T"], case["E"]
        logits = 2.0 * torch.randn((T, E), generator=gen, device=DEV)
        if case["masked"]:
            hole = torch.rand((T, E), generator=gen, device=DEV) < 0.2
            logits = logits.masked_fill(hole, float("-inf"))
            logits[T - T // 16:] = float("-inf")
        st["logits"] = logits.to(DTYPES[case["dtype"]])
        st["bias"] = 0.1 * torch.randn(E, generator=gen, device=DEV) if case["bias"] else None
        return st
    dt = DTYPES[case["dtype"]]
    if op == "w4":
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        st["q"] = torch.empty((N, K // 2), dtype=torch.uint8, device=DEV)
        c = _codes(gen, (N, K), 7.5, 3.2, 0, 15)
        st["q"].copy_(c[:, 0::2] | (c[:, 1::2] << 4))
        spread = 0.02 * (0.6 + 0.8 * torch.rand((N, K // G), generator=gen, device=DEV))
        st["scales"] = (spread / 3.2).to(DTYPES[case["sdtype"]])
        st["zeros"] = (torch.randint(5, 11, (N, K // G), generator=gen, device=DEV, dtype=torch.int32).to(torch.uint8)
                       if case["zeros"] else None)
        st["x"] = torch.randn((M, K), generator=gen, device=DEV).to(dt)
        return st
    T, E, k, N, K = case["T"], case["E"], case["k"], case["N"], case["K"]
    fmt = case["fmt"]
    st["w"] = [_blocks(gen, fmt, E * N, K).view(E, N, -1) for _ in range(2 if op == "glu" else 1)]
    st["ids"], st["weights"] = _choices(gen, T, E, k, case["pad"])
    shape = (T, k, K) if op == "combine" else (T, K)
    st["x"] = torch.randn(shape, generator=gen, device=DEV).to(dt)
    return st


# -------------------------------------------------------------- plain form ---

def _dequant(fmt, w, K):
    """f32 rows of GGUF blocks (uint8 [..., bytes])."""
    qk, qb = BLOCK[fmt]
    b = w.reshape(*w.shape[:-1], K // qk, qb)
    if fmt in ("Q8_0", "Q4_0", "Q5_0"):
        d = b[..., :2].contiguous().view(torch.float16).float()
        if fmt == "Q8_0":
            v = b[..., 2:].contiguous().view(torch.int8).float()
        else:
            qs = b[..., -16:]
            v = torch.cat([qs & 15, qs >> 4], -1).float()
            if fmt == "Q5_0":
                sh = torch.arange(8, device=w.device, dtype=torch.uint8)
                v = v + 16.0 * ((b[..., 2:6, None] >> sh) & 1).flatten(-2).float()
            v = v - (8.0 if fmt == "Q4_0" else 16.0)
        return (v * d).flatten(-2)
    if fmt == "Q4_K":
        d = b[..., 0:2].contiguous().view(torch.float16).float()
        dmin = b[..., 2:4].contiguous().view(torch.float16).float()
        a, c, e = b[..., 4:8], b[..., 8:12], b[..., 12:16]
        sc = torch.cat([a & 63, (e & 15) | ((a >> 6) << 4)], -1).float()
        mn = torch.cat([c & 63, (e >> 4) | ((c >> 6) << 4)], -1).float()
        qs = b[..., 16:].unflatten(-1, (4, 32))
        q = torch.stack([qs & 15, qs >> 4], -2).flatten(-3, -2).float()  # [..., 8, 32]
        return ((d * sc)[..., None] * q - (dmin * mn)[..., None]).flatten(-3)
    ql = b[..., :128].unflatten(-1, (2, 2, 32))
    qh = b[..., 128:192].unflatten(-1, (2, 32))
    sc = b[..., 192:208].contiguous().view(torch.int8).float()
    d = b[..., 208:].contiguous().view(torch.float16).float()
    q = torch.stack([(ql[..., 0, :] & 15) | ((qh & 3) << 4), (ql[..., 1, :] & 15) | (((qh >> 2) & 3) << 4),
                     (ql[..., 0, :] >> 4) | (((qh >> 4) & 3) << 4), (ql[..., 1, :] >> 4) | ((qh >> 6) << 4)], -2)
    q = q.flatten(-3).float().unflatten(-1, (16, 16)) - 32.0
    return ((d * sc)[..., None] * q).flatten(-3)


def _plain_route(st):
    c = st["case"]
    l = st["logits"].double()
    T, E = l.shape
    dead = torch.isnan(l) | (l == float("-inf"))
    if c["score"] == "softmax":
        top = l.masked_fill(dead, float("-inf")).amax(1, keepdim=True)
        ex = torch.where(dead, torch.zeros_like(l), torch.exp(l - top))
        s = ex / ex.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    choice = s if st["bias"] is None else s + st["bias"].double()
    choice = choice.masked_fill(dead, float("-inf"))
    if c["groups"] > 1:
        g = choice.view(T, c["groups"], -1)
        best = torch.sort(g, dim=2, descending=True).values[..., :c["group_top"]]
        alive = best[..., 0] > float("-inf")
        gs = best.masked_fill(best == float("-inf"), 0.0).sum(-1).masked_fill(~alive, float("-inf"))
        order = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, order, True)
        choice = choice.masked_fill(~keep.repeat_interleave(E // c["groups"], 1), float("-inf"))
    v, i = torch.sort(choice, dim=1, descending=True, stable=True)
    v, i = v[:, :c["k"]], i[:, :c["k"]]
    none = v == float("-inf")
    w = s.gather(1, i).masked_fill(none, 0.0)
    if c["renorm"]:
        w = torch.where(w.sum(1, keepdim=True) > 0, w / w.sum(1, keepdim=True), torch.zeros_like(w))
    return i.masked_fill(none, -1).to(torch.int32), (w * c["scale"]).float()


def _plain_products(st, per_slot):
    """f32 products [mats][T, k, N] of each token's slots with their experts' rows."""
    c = st["case"]
    ids, x = st["ids"], st["x"]
    T, k, N, K = c["T"], c["k"], c["N"], c["K"]
    rows = x.float().reshape(-1, K) if per_slot else x.float().repeat_interleave(k, 0)
    flat = ids.reshape(-1)
    outs = [torch.zeros((T * k, N), device=x.device) for _ in st["w"]]
    if T * k * N * K <= 1 << 26:
        live = ((flat >= 0) & (flat < c["E"])).float()[:, None]
        for o, w in zip(outs, st["w"]):
            wd = _dequant(c["fmt"], w[flat.clamp(0, c["E"] - 1).long()], K)
            o.copy_((wd * rows[:, None, :]).sum(-1) * live)
    else:
        for e in range(c["E"]):
            sel = (flat == e).nonzero()[:, 0]
            if sel.numel():
                xe = rows[sel]
                for o, w in zip(outs, st["w"]):
                    o[sel] = xe @ _dequant(c["fmt"], w[e], K).t()
    return [o.view(T, k, N) for o in outs]


def _plain_act(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    t = 0.7978845608028654 * (v + 0.044715 * v * v * v)
    return v / (1.0 + torch.exp(-2.0 * t))


def _plain(st):
    op, c = st["op"], st["case"]
    if op == "route":
        return _plain_route(st)
    dt = DTYPES[c["dtype"]]
    if op == "w4":
        q = st["q"]
        codes = torch.stack([q & 15, q >> 4], -1).flatten(1).float().unflatten(1, (-1, c["G"]))
        z = 8.0 if st["zeros"] is None else st["zeros"].float()[..., None]
        w = ((codes - z) * st["scales"].float()[..., None]).flatten(1)
        return (st["x"].float() @ w.t()).to(dt)
    if op == "matmul":
        return _plain_products(st, False)[0].to(dt)
    if op == "glu":
        g, u = _plain_products(st, False)
        return (_plain_act(g, c["act"]) * u).to(dt)
    y = _plain_products(st, True)[0]
    return (y * st["weights"][..., None]).sum(1).to(dt)


# ---------------------------------------------------------------- own form ---

def _own(st):
    import block_quantized_matmul_gguf_amd as qmm

    op, c = st["op"], st["case"]
    if op == "route":
        return qmm.route_experts(st["logits"], c["k"], score=c["score"], bias=st["bias"], groups=c["groups"],
                                 top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renorm"],
                                 scale=c["scale"])
    if op == "w4":
        return qmm.w4_matmul(st["q"], st["scales"], st["x"], zeros=st["zeros"])
    fmt = FMT_ID[c["fmt"]]
    if op == "matmul":
        return qmm.experts_matmul(fmt, st["w"][0], st["x"], st["ids"])
    if op == "glu":
        return qmm.experts_glu(fmt, st["w"][0], st["w"][1], st["x"], st["ids"], act=c["act"])
    return qmm.experts_combine(fmt, st["w"][0], st["x"], st["ids"], st["weights"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- exact ---

def _exact_rows(fmt, w, K):
    """f64 rows, element by element: where element k of a row has its bits, its scale and its offset."""
    qk, qb = BLOCK[fmt]
    k = torch.arange(K, device=w.device)
    base, j = (k // qk) * qb, k % qk

    def byte(off):
        return w[:, off].long()

    def half(off):
        lo, hi = byte(off), byte(off + 1)
        return (lo | (hi << 8)).to(torch.int16).view(torch.float16).double()

    def signed(v):
        return torch.where(v > 127, v - 256, v).double()

    if fmt == "Q8_0":
        return half(base) * signed(byte(base + 2 + j))
    if fmt == "Q4_0":
        return half(base) * (((byte(base + 2 + j % 16) >> (4 * (j // 16))) & 15) - 8).double()
    if fmt == "Q5_0":
        low = (byte(base + 6 + j % 16) >> (4 * (j // 16))) & 15
        fifth = (byte(base + 2 + j // 8) >> (j % 8)) & 1
        return half(base) * (low + 16 * fifth - 16).double()
    if fmt == "Q4_K":
        s = j // 32
        early = s < 4
        a, b = byte(base + 4 + s % 4), byte(base + 8 + s % 4)
        e = byte(base + 12 + s % 4)
        sc = torch.where(early, a & 63, (e & 15) | ((a >> 6) << 4)).double()
        mn = torch.where(early, b & 63, (e >> 4) | ((b >> 6) << 4)).double()
        q = ((byte(base + 16 + 32 * (s // 2) + j % 32) >> (4 * (s % 2))) & 15).double()
        return half(base) * sc * q - half(base + 2) * mn
    h, r = j // 128, j % 128
    low = (byte(base + 64 * h + r % 64) >> (4 * (r // 64))) & 15
    high = (byte(base + 128 + 32 * h + r % 32) >> (2 * (r // 32))) & 3
    return half(base + 208) * signed(byte(base + 192 + j // 16)) * (low + 16 * high - 32).double()


def _exact_route(case, st):
    l = st["logits"].double().cpu().tolist()
    bias = [0.0] * case["E"] if st["bias"] is None else st["bias"].double().cpu().tolist()
    size = case["E"] // case["groups"]
    weights = []
    for row in l:
        live = [e for e, v in enumerate(row) if v == v and v != -math.inf]
        if case["score"] == "softmax":
            top = max((row[e] for e in live), default=0.0)
            part = {e: math.exp(row[e] - top) for e in live}
            total = math.fsum(part.values())
            s = {e: part[e] / total for e in live}
        else:
            s = {e: 1.0 / (1.0 + math.exp(-row[e])) for e in live}
        choice = {e: s[e] + bias[e] for e in live}
        if case["groups"] > 1:
            score = {}
            for e in live:
                score.setdefault(e // size, []).append(choice[e])
            ranked = sorted(score, key=lambda g: (-sum(sorted(score[g], reverse=True)[:case["group_top"]]), g))
            kept = set(ranked[:case["top_groups"]])
            choice = {e: v for e, v in choice.items() if e // size in kept}
        ids = sorted(choice, key=lambda e: (-choice[e], e))[:case["k"]]
        w = [s[e] for e in ids]
        if case["renorm"]:
            total = math.fsum(w)
            w = [v / total if total > 0 else 0.0 for v in w]
        weights.append([v * case["scale"] for v in w] + [0.0] * (case["k"] - len(w)))
    return None, torch.tensor(weights, dtype=torch.float64, device=DEV)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    x = st["x"].double()
    if op == "w4":
        k = torch.arange(case["K"], device=DEV)
        grp = k // case["G"]
        y = torch.empty((case["M"], case["N"]), dtype=torch.float64, device=DEV)
        for n in range(0, case["N"], 2048):
            code = (st["q"][n:n + 2048][:, k // 2].long() >> (4 * (k % 2))) & 15
            zero = 8 if st["zeros"] is None else st["zeros"][n:n + 2048].long()[:, grp]
            y[:, n:n + 2048] = x @ ((code - zero).double() * st["scales"][n:n + 2048].double()[:, grp]).t()
        return y
    T, k, N = case["T"], case["k"], case["N"]
    xr = x.view(T * k, -1) if op == "combine" else x
    flat = st["ids"].view(-1)
    slots = [torch.zeros((T * k, N), dtype=torch.float64, device=DEV) for _ in st["w"]]
    for e in torch.unique(flat).tolist():
        if e < 0:
            continue
        at = (flat == e).nonzero()[:, 0]
        src = at if op == "combine" else at // k
        for out, w in zip(slots, st["w"]):
            for n in range(0, N, 1024):
                out[at, n:n + 1024] = xr[src] @ _exact_rows(case["fmt"], w[e, n:n + 1024], case["K"]).t()
    if op == "matmul":
        return slots[0].view(T, k, N)
    if op == "glu":
        g, u = slots
        if case["act"] == "silu":
            h = g / (1.0 + torch.exp(-g)) * u
        else:
            h = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))) * u
        return h.view(T, k, N)
    return (slots[0].view(T, k, N) * st["weights"].double()[..., None]).sum(1)
