"""Cases that time the quantized paged cache of keys and values: writing it, reading it back, attention over it.

``own = False`` computes each operator in elementary torch operations; ``own = True`` calls the package.  ``exact``
computes the same outputs in 64 bits from the definitions, apart from the plain form.

Operators:
  store      new tokens' keys and values quantized into the pages of their sequences, then read back
  load       keys and values of whole sequences read back from their pages
  attention  softmax(scale q . k) v of new tokens (one or many per sequence) over the pages of their sequence

A cache is uint8 [pages, heads, page size, row bytes]; the bytes of 64 neighbouring tokens of a head hold their codes
in the order in which matrix instructions take them, then their scales:
  * a token is t = 16 u + 4 g + i = 32 s + 16 h + 4 g + i, a dimension d = 32 b + 8 c + e = 32 b + 16 p + n; a
    quantized block is the 32 dimensions of b;
  * the scales are f16 [D / 32][64], token t at place 16 g + 8 s + 4 h + i;
  * keys: four tiles (u) of 64 lanes (16 c + t % 16); a lane holds the codes of its eight dimensions of every b, cut
    into pieces of 16 bytes (and a rest), each piece as [64 lanes][bytes];
  * values: per b 64 lanes (16 g + n); a lane holds 16 tokens (8 s + 4 h + i); Q8_0 [p][lane][16 bytes], Q4_0
    [lane][p][8 bytes];
  * Q8_0 codes are bytes q + 128; of eight Q4_0 codes, number e is nibble e / 2 + 4 (e % 2) of a 32-bit word.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
FMT_ID = {"Q4_0": 2, "Q8_0": 8}
ROW = {"Q4_0": 18, "Q8_0": 34}  # bytes per 32 values
GROUP = 64                      # tokens whose bytes lie together


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one token of one chat appended to a small model's cache: launch latency
        dict(name="store_1_q8_3x64", op="store", B=1, L=307, new=1, ragged=False, H=3, D=64, page=64, fk="Q8_0", fv="Q8_0",
             dtype="f32"),
        # a decoding batch: one token of each of 64 sequences
        dict(name="store_64x1_q8_8x128", op="store", B=64, L=4096, new=1, ragged=True, H=8, D=128, page=64, fk="Q8_0",
             fv="Q8_0", dtype="bf16"),
        # prompts of different lengths, values in 4 bits
        dict(name="store_8k_q8q4_8x128", op="store", B=5, L=2600, new=0, ragged=True, H=8, D=128, page=128, fk="Q8_0",
             fv="Q4_0", dtype="bf16"),
        # one short sequence read back
        dict(name="load_307_q8_3x64", op="load", B=1, L=307, new=0, ragged=False, H=3, D=64, page=64, fk="Q8_0", fv="Q8_0",
             dtype="f32"),
        # several long sequences read back, to move or to check them
        dict(name="load_64k_q4_8x128", op="load", B=7, L=14000, new=0, ragged=True, H=8, D=128, page=256, fk="Q4_0",
             fv="Q4_0", dtype="f16"),
        # the next token of one chat with a small model: launch latency
        dict(name="attn_1x307_q8_9_3x64", op="attention", B=1, L=307, new=1, ragged=False, H=3, G=3, D=64, page=64,
             fk="Q8_0", fv="Q8_0", dtype="f32", causal=True, window=0, softcap=0.0),
        # a decoding batch of uneven lengths: bandwidth
        dict(name="attn_64x1_8k_q8_32_8x128", op="attention", B=64, L=8192, new=1, ragged=True, H=8, G=4, D=128, page=64,
             fk="Q8_0", fv="Q8_0", dtype="bf16", causal=True, window=0, softcap=0.0),
        # one token over a very long context in 4 bits: the work split along it
        dict(name="attn_1x128k_q4_32_8x128", op="attention", B=1, L=131072, new=1, ragged=False, H=8, G=4, D=128, page=256,
             fk="Q4_0", fv="Q4_0", dtype="f16", causal=True, window=0, softcap=0.0),
        # drafted tokens checked together, wide heads, a sliding window and capped scores
        dict(name="attn_16x5_win_q8q4_8_4x256", op="attention", B=16, L=4000, new=5, ragged=True, H=4, G=2, D=256, page=128,
             fk="Q8_0", fv="Q4_0", dtype="bf16", causal=True, window=1024, softcap=50.0),
        # a whole prompt of a small model
        dict(name="attn_307_q8_9_3x64", op="attention", B=1, L=307, new=307, ragged=False, H=3, G=3, D=64, page=64,
             fk="Q8_0", fv="Q8_0", dtype="f32", causal=True, window=0, softcap=0.0),
        # chunks of several prompts beside each other, a key head for each query head
        dict(name="attn_6x300_q8_8_8x96", op="attention", B=6, L=3500, new=300, ragged=True, H=8, G=1, D=96, page=64,
             fk="Q8_0", fv="Q8_0", dtype="f16", causal=True, window=0, softcap=0.0),
        # a chunk of a long prompt: matrix rate
        dict(name="attn_2048_10k_q8_32_8x128", op="attention", B=1, L=10240, new=2048, ragged=False, H=8, G=4, D=128,
             page=128, fk="Q8_0", fv="Q8_0", dtype="bf16", causal=True, window=0, softcap=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "load", "attention", "attention", "attention"])
    case = dict(op=op, H=rng.choice([1, 2, 3, 4, 8]), D=rng.choice([64, 96, 128, 256]), page=rng.choice([64, 128, 256]),
                fk=rng.choice(["Q8_0", "Q4_0"]), fv=rng.choice(["Q8_0", "Q4_0"]), dtype=rng.choice(["f32", "f16", "bf16"]))
    B = _log(rng, 1, 64)
    L = _log(rng, 1, 65536)
    row = case["H"] * case["D"]
    if op != "attention":
        while B * L * row > 64000 * 8 * 128:
            B, L = (B + 1) // 2, (L + 1) // 2
        new = 0 if op == "load" or rng.random() < 0.5 else min(L, _log(rng, 1, 64))
        case.update(B=B, L=L, new=new, ragged=rng.random() < 0.7)
        return case
    case["G"] = rng.choice([1, 2, 3, 4, 6, 8])
    if rng.random() < 0.3:
        case["G"] = 1
    new = min(L, _log(rng, 1, 2048)) if rng.random() < 0.6 else 1
    while B * L * row > 64 * 4096 * 8 * 128 or B * L * new * row * case["G"] > 2048 * 8192 * 32 * 128:
        B, L = (B + 1) // 2, (L + 1) // 2
        new = min(new, L)
    case.update(B=B, L=L, new=new, ragged=rng.random() < 0.7, causal=rng.random() < 0.85, window=0, softcap=0.0)
    if case["causal"] and rng.random() < 0.25:
        case["window"] = _log(rng, 1, 4096)
    if rng.random() < 0.2:
        case["softcap"] = rng.choice([20.0, 50.0])
    return case


def _sizes(case):
    """(lengths, new tokens) of the sequences: the length counts the new tokens."""
    r = random.Random(case["B"] * 1000003 + case["L"] * 101 + case["new"])
    lengths, new = [], []
    for s in range(case["B"]):
        n = case["L"] if not case["ragged"] or s == 0 else r.randint(max(1, case["L"] // 8), case["L"])
        m = n if case["new"] == 0 else min(n, case["new"])
        if case["ragged"] and s and case["new"] > 1:
            m = r.randint(1, m)
        lengths.append(n)
        new.append(m)
    return lengths, new


def _seen(case):
    """Per sequence: positions that any new token sees, and pairs of a new token and a position it sees."""
    spans, pairs = [], []
    for n, m in zip(*_sizes(case)):
        if not case["causal"]:
            spans.append(n)
            pairs.append(n * m)
            continue
        w = case["window"] or n
        pairs.append(sum(min(w, n - m + i + 1) for i in range(m)))
        spans.append(min(n, w + m - 1))
    return spans, pairs


def work(case):
    H, D, e = case["H"], case["D"], SIZE[case["dtype"]]
    token = H * (D // 32) * (ROW[case["fk"]] + ROW[case["fv"]])  # cache bytes of a token
    lengths, new = _sizes(case)
    if case["op"] == "store":  # read the new tokens, write them, read them back, write the values
        return {"bytes": sum(new) * (2 * token + 4 * H * D * e), "flops": 8 * sum(new) * H * D}
    if case["op"] == "load":
        return {"bytes": sum(lengths) * (token + 2 * H * D * e), "flops": 2 * sum(lengths) * H * D}
    spans, pairs = _seen(case)
    heads = H * case["G"]
    return {"bytes": sum(spans) * token + 2 * sum(new) * heads * D * e, "flops": 4 * sum(pairs) * heads * D}


# ----------------------------------------------------------------- layout ---

def _places(fmt, values, D):
    """Where a group of 64 tokens has its codes: byte [64, D], shift [64, D], and its scales: byte [64, D / 32]."""
    t = torch.arange(GROUP, device=DEV)[:, None]
    d = torch.arange(D, device=DEV)[None, :]
    g, s, h, i = (t >> 2) & 3, t >> 5, (t >> 4) & 1, t & 3
    b = d >> 5
    if values:
        lane, e, p = 16 * g + (d & 15), 4 * h + i, (d >> 4) & 1
        if fmt == "Q8_0":
            byte, shift = 2048 * b + 1024 * p + 16 * lane + 8 * s + e, torch.zeros_like(t + d)
        else:
            nib = (e >> 1) + 4 * (e & 1)
            byte, shift = 1024 * b + 16 * lane + 8 * p + 4 * s + (nib >> 1), 4 * (nib & 1) + 0 * d
    else:
        lane, e = 16 * ((d >> 3) & 3) + (t & 15), d & 7
        if fmt == "Q8_0":
            held, at, shift = D // 4, 8 * b + e, torch.zeros_like(t + d)
        else:
            nib = (e >> 1) + 4 * (e & 1)
            held, at, shift = D // 8, 4 * b + (nib >> 1), 4 * (nib & 1) + 0 * t
        piece = at >> 4
        size = (held - 16 * piece).clamp(max=16)  # bytes a lane holds of this piece
        byte = (t >> 4) * 64 * held + 1024 * piece + lane * size + (at & 15)
    codes = GROUP * D if fmt == "Q8_0" else GROUP * D // 2
    place = 16 * g + 8 * s + 4 * h + i
    scale = codes + 2 * (64 * torch.arange(D // 32, device=DEV)[None, :] + place)
    return byte, shift, scale


def _quantize(fmt, x):
    """Codes int32 [..., D] (as stored) and f16 scales [..., D / 32] of f32 values."""
    v = x.unflatten(-1, (-1, 32))
    mag = v.abs()
    top, at = mag.max(-1, keepdim=True)
    if fmt == "Q8_0":
        d = top / 127.0
    else:
        at = (mag == top).to(torch.int32).argmax(-1, keepdim=True)  # the first of the largest
        d = v.gather(-1, at) / -8.0
    d16 = d.to(torch.float16)
    dead = ~torch.isfinite(mag).all(-1, keepdim=True) | ~torch.isfinite(d16)
    none = dead | (d16 == 0)
    y = v * torch.where(none, torch.zeros_like(d), 1.0 / d)
    if fmt == "Q8_0":
        whole = torch.trunc(y)
        q = whole + torch.sign(y) * ((y - whole).abs() >= 0.5) + 128.0
    else:
        q = torch.trunc(y + 8.5).clamp(max=15.0)
    q = torch.where(none, torch.full_like(q, 128.0 if fmt == "Q8_0" else 8.0), q)
    d16 = torch.where(dead, torch.full_like(d16, float("nan")), d16)
    return q.flatten(-2).to(torch.int32), d16[..., 0]


def _pack(fmt, values, x):
    """Cache bytes of whole groups: f32 [..., 64, D] -> uint8 [..., 64 * row bytes]."""
    D = x.shape[-1]
    byte, shift, scale = _places(fmt, values, D)
    q, d = _quantize(fmt, x)
    out = torch.zeros((*x.shape[:-2], GROUP * D // 32 * ROW[fmt]), dtype=torch.int32, device=x.device)
    out.index_add_(-1, byte.flatten(), (q << shift.to(torch.int32)).flatten(-2))
    raw = d.contiguous().view(torch.uint8).view(*d.shape, 2).to(torch.int32)
    out[..., scale.flatten()] = raw[..., 0].flatten(-2)
    out[..., scale.flatten() + 1] = raw[..., 1].flatten(-2)
    return out.to(torch.uint8)


def _unpack(fmt, values, group, D):
    """f32 values [..., 64, D] of groups of cache bytes [..., 64 * row bytes]."""
    byte, shift, scale = _places(fmt, values, D)
    q = group[..., byte]
    q = q.float() - 128.0 if fmt == "Q8_0" else ((q >> shift.to(torch.uint8)) & 15).float() - 8.0
    raw = torch.stack([group[..., scale], group[..., scale + 1]], -1)
    return (q.unflatten(-1, (-1, 32)) * raw.view(torch.float16).float()).flatten(-2)


# ----------------------------------------------------------------- inputs ---

def _fill(gen, case, pages, fmt, values, spread):
    """A pool of pages as earlier tokens left it."""
    H, D, page = case["H"], case["D"], case["page"]
    pool = torch.empty((pages, H, page, D // 32 * ROW[fmt]), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (H * page * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn((n, H, page // GROUP, GROUP, D), generator=gen, device=DEV) * spread
        pool[p:p + n] = _pack(fmt, values, x).view(n, H, page, -1)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    H, D, page = case["H"], case["D"], case["page"]
    lengths, new = _sizes(case)
    held = [-(-n // page) for n in lengths]
    pages = sum(held) + 2
    spread = 0.7 + 0.3 * torch.rand(D, generator=gen, device=DEV)
    spread = torch.where(torch.rand(D, generator=gen, device=DEV) < 0.03, 4.0 * spread, spread)  # keys have wide channels
    st = {"case": case, "lengths_h": lengths, "new_h": new}
    st["k_cache"] = _fill(gen, case, pages, case["fk"], False, spread)
    st["v_cache"] = _fill(gen, case, pages, case["fv"], True, 1.0)
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((case["B"], max(held)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(held):
        table[s, :n] = order[at:at + n]
        at += n
    st["table"] = table
    st["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    counts = lengths if case["op"] == "load" else new
    st["starts"] = torch.tensor([sum(counts[:s]) for s in range(case["B"] + 1)], dtype=torch.int32, device=DEV)
    st["tokens"] = sum(counts)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "store":
        st["k"] = (torch.randn((sum(new), H, D), generator=gen, device=DEV) * spread).to(dt)
        st["v"] = torch.randn((sum(new), H, D), generator=gen, device=DEV).to(dt)
    elif case["op"] == "attention":
        st["q"] = (1.3 * torch.randn((sum(new), H * case["G"], D), generator=gen, device=DEV)).to(dt)
    return st


# -------------------------------------------------------------- plain form ---

def _positions(st):
    """Sequence and position of each of the tokens that starts counts."""
    n = torch.arange(st["tokens"], device=DEV)
    seq = (n[:, None] >= st["starts"][None, 1:]).sum(1)
    behind = st["starts"].long()[seq + 1] - n
    return seq, st["lengths"].long()[seq] - behind


def _plain_store(st):
    c = st["case"]
    H, D, page = c["H"], c["D"], c["page"]
    seq, pos = _positions(st)
    at = st["table"][seq, pos // page].long()
    group, t = pos % page // GROUP, pos % GROUP
    heads = torch.arange(H, device=DEV)[None, :, None]
    for fmt, values, cache, x in ((c["fk"], False, st["k_cache"], st["k"]), (c["fv"], True, st["v_cache"], st["v"])):
        byte, shift, scale = _places(fmt, values, D)
        flat = cache.view(cache.shape[0], H, page // GROUP, -1)
        q, d = _quantize(fmt, x.float())
        where = (at[:, None, None], heads, group[:, None, None])
        if fmt == "Q8_0":
            flat[(*where, byte[t][:, None])] = q.to(torch.uint8)
        elif values:  # neighbouring tokens share a byte, one of them in its low half
            for half in (0, 4):
                mine = shift[t, 0] == half
                w = (at[mine][:, None, None], heads, group[mine][:, None, None], byte[t[mine]][:, None])
                flat[w] = (flat[w] & (0xF0 >> half)) | (q[mine] << half).to(torch.uint8)
        else:
            order = torch.argsort(byte[0] * 8 + shift[0])
            low, high = order[0::2], order[1::2]
            flat[(*where, byte[t][:, None][..., low])] = (q[..., low] | (q[..., high] << 4)).to(torch.uint8)
        raw = d.contiguous().view(torch.uint8).view(*d.shape, 2)
        flat[(*where, scale[t][:, None])] = raw[..., 0]
        flat[(*where, scale[t][:, None] + 1)] = raw[..., 1]
    return _plain_load(st)


def _plain_load(st):
    c = st["case"]
    H, D, page = c["H"], c["D"], c["page"]
    seq, pos = _positions(st)
    at = st["table"][seq, pos // page].long()
    group, t = pos % page // GROUP, pos % GROUP
    heads = torch.arange(H, device=DEV)[None, :, None]
    out = []
    for fmt, values, cache in ((c["fk"], False, st["k_cache"]), (c["fv"], True, st["v_cache"])):
        byte, shift, scale = _places(fmt, values, D)
        flat = cache.view(cache.shape[0], H, page // GROUP, -1)
        where = (at[:, None, None], heads, group[:, None, None])
        q = flat[(*where, byte[t][:, None])]
        if fmt == "Q8_0":
            q = q.float() - 128.0
        else:
            q = ((q >> shift[t][:, None].to(torch.uint8)) & 15).float() - 8.0
        raw = torch.stack([flat[(*where, scale[t][:, None])], flat[(*where, scale[t][:, None] + 1)]], -1)
        d = raw.view(torch.float16).float()
        out.append((q.unflatten(-1, (-1, 32)) * d).flatten(-2).to(DTYPES[c["dtype"]]))
    return out


def _plain_attention(st):
    c = st["case"]
    H, G, D, page, B = c["H"], c["G"], c["D"], c["page"], c["B"]
    most = max(st["new_h"])
    pages = st["table"].clamp_min(0).long()
    k, v = (_unpack(fmt, values, cache[pages].view(*pages.shape, H, page // GROUP, -1), D)
            .permute(0, 2, 1, 3, 4, 5).reshape(B, H, -1, D)
            for fmt, values, cache in ((c["fk"], False, st["k_cache"]), (c["fv"], True, st["v_cache"])))
    starts, lengths = st["starts"].long(), st["lengths"].long()
    i = torch.arange(most, device=DEV)
    count = starts[1:] - starts[:-1]
    live = i[None, :] < count[:, None]
    rows = (starts[:-1, None] + i[None, :]).clamp(max=st["tokens"] - 1)
    q = st["q"].float()[rows].view(B, most, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * most, D)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()) / math.sqrt(D)
    if c["softcap"]:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    j = torch.arange(k.shape[2], device=DEV)
    pos = lengths[:, None] - count[:, None] + i[None, :]
    gone = j[None, None, :] >= lengths[:, None, None]
    if c["causal"]:
        gone = gone | (j[None, None, :] > pos[:, :, None])
    if c["window"]:
        gone = gone | (j[None, None, :] <= pos[:, :, None] - c["window"])
    s = s.view(B, H, G, most, -1).masked_fill_(gone[:, None, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p.view(B, H, G * most, -1), v) / p.sum(-1).view(B, H, G * most, 1)
    o = o.view(B, H, G, most, D).permute(0, 3, 1, 2, 4).reshape(B, most, H * G, D)
    return o[live].to(DTYPES[c["dtype"]])


# ---------------------------------------------------------------- own form ---

def _own(st):
    import block_quantized_matmul_gguf_amd as qmm

    c = st["case"]
    cache = (FMT_ID[c["fk"]], FMT_ID[c["fv"]], st["k_cache"], st["v_cache"])
    batch = (st["table"], st["starts"], st["lengths"])
    if c["op"] == "attention":
        return qmm.cache_attention(*cache, st["q"], *batch, causal=c["causal"], window=c["window"], softcap=c["softcap"],
                                   max_length=c["L"])
    if c["op"] == "store":
        qmm.cache_store(*cache, st["k"], st["v"], *batch)
    return list(qmm.cache_load(*cache, *batch, tokens=st["tokens"], dtype=DTYPES[c["dtype"]]))


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_attention(state) if op == "attention" else _plain_store(state) if op == "store" else _plain_load(state)


# ------------------------------------------------------------------- exact ---

def _exact_quantize(fmt, x):
    """f64 values of the blocks that numpy's f32 steps of the formats' rule give for x."""
    import numpy as np

    v = x.float().cpu().numpy().reshape(-1, 32)
    one = np.float32(1.0)
    mag = np.abs(v)
    first = mag.argmax(1)
    if fmt == "Q8_0":
        d = (mag[np.arange(len(v)), first] / np.float32(127.0)).astype(np.float32)
    else:
        d = (v[np.arange(len(v)), first] / np.float32(-8.0)).astype(np.float32)
    half = d.astype(np.float16)
    inv = np.divide(one, d, out=np.zeros_like(d), where=half != 0)
    y = (v * inv[:, None]).astype(np.float32)
    if fmt == "Q8_0":
        q = np.copysign(np.floor(np.abs(y.astype(np.float64)) + 0.5), y)
    else:
        q = np.minimum(np.floor((y + np.float32(8.5)).astype(np.float64)), 15.0) - 8.0
    return torch.from_numpy((q * half.astype(np.float64)[:, None]).reshape(x.shape)).to(DEV)


def _exact_rows(fmt, values, raw, D):
    """f64 [heads, tokens, D] of whole groups, their bytes [heads, bytes] end to end, dimension by dimension."""
    size = GROUP * (D // 32) * ROW[fmt]
    n = raw.shape[1] // size * GROUP
    t = torch.arange(n, device=DEV)
    base, t = t // GROUP * size, t % GROUP
    quad, pair, low = t % 16 // 4, t // 32, t % 32 // 16 * 4 + t % 4  # 4 tokens in a row, which 32, which of 8
    out = torch.empty((raw.shape[0], n, D), dtype=torch.float64, device=DEV)
    for d in range(D):
        b, r = divmod(d, 32)
        if fmt == "Q8_0":
            if values:
                at = b * 2048 + r // 16 * 1024 + (quad * 16 + r % 16) * 16 + pair * 8 + low
            else:
                whole, rest = divmod(D // 4, 16)
                piece, off = divmod(8 * b + r % 8, 16)
                at = t // 16 * (16 * D) + piece * 1024 + (r // 8 * 16 + t % 16) * (16 if piece < whole else rest) + off
            code = raw[:, base + at].long() - 128
        else:
            if values:
                nib = low // 2 + low % 2 * 4
                at = b * 1024 + (quad * 16 + r % 16) * 16 + r // 16 * 8 + pair * 4 + nib // 2
            else:
                nib = torch.full_like(t, r % 8 // 2 + r % 2 * 4)
                whole, rest = divmod(D // 8, 16)
                word, off = divmod(4 * b, 16)
                at = t // 16 * (8 * D) + word * 1024 + (r // 8 * 16 + t % 16) * (16 if word < whole else rest) + off + nib // 2
            code = (raw[:, base + at].long() >> (nib % 2 * 4)) % 16 - 8
        at = base + size - 128 * (D // 32) + 128 * b + 2 * (quad * 16 + pair * 8 + low)
        bits = raw[:, at].to(torch.int32) + 256 * raw[:, at + 1].to(torch.int32)
        out[:, :, d] = code.double() * bits.to(torch.int16).view(torch.float16).double()
    return out


def _exact_sequence(st, fmt, values, cache, s):
    c = st["case"]
    n = st["lengths_h"][s]
    ids = st["table"][s, :-(-n // c["page"])].long()
    return _exact_rows(fmt, values, cache[ids].transpose(0, 1).reshape(c["H"], -1), c["D"])[:, :n]


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "store":
        return [_exact_quantize(c["fk"], st["k"]), _exact_quantize(c["fv"], st["v"])]
    lengths, new = _sizes(c)
    if sum(_seen(c)[1] if c["op"] == "attention" else [0]) * c["H"] * c.get("G", 1) * c["D"] > 1 << 41:
        return None
    kinds = ((c["fk"], False, st["k_cache"]), (c["fv"], True, st["v_cache"]))
    if c["op"] == "load":
        return [torch.cat([_exact_sequence(st, *kind, s).transpose(0, 1) for s in range(c["B"])]) for kind in kinds]
    scale = 1.0 / math.sqrt(c["D"])
    rows, at = [], 0
    for s, (n, m) in enumerate(zip(lengths, new)):
        out = torch.empty((m, c["H"] * c["G"], c["D"]), dtype=torch.float64, device=DEV)
        place = torch.arange(n - m, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None, :]
        seen = torch.ones((m, n), dtype=torch.bool, device=DEV)
        if c["causal"]:
            seen = j <= place
        if c["window"]:
            seen = seen & (place - j < c["window"])
        k, v = (_exact_sequence(st, *kind, s) for kind in kinds)
        for h in range(c["H"]):
            for g in range(c["G"]):
                x = st["q"][at:at + m, h * c["G"] + g].double() @ k[h].t().contiguous() * scale
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                x = torch.where(seen, x, torch.full_like(x, float("-inf")))
                out[:, h * c["G"] + g] = torch.softmax(x, 1) @ v[h]
        rows.append(out)
        at += m
    return torch.cat(rows)
