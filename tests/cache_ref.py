"""The quantized paged cache in numpy, from its definition: GGUF blocks of the
oracle's quantizers, the place of each code and scale, and attention in 64 bits."""
import numpy as np

import oracle

Q4_0, Q8_0 = 2, 8
BLOCK = {Q4_0: 18, Q8_0: 34}


def row_bytes(fmt, dim):
    return dim // 32 * BLOCK[fmt]


def quantize(fmt, x):
    """f32 [..., D] -> (codes int [..., D] as signed values, scales f16 [..., D / 32]) by the oracle's GGUF blocks,
    with the cache's two exceptions (a scale of 0: codes 0; not finite: NaN)."""
    shape, dim = x.shape[:-1], x.shape[-1]
    flat = np.ascontiguousarray(x.reshape(-1, dim), dtype=np.float32)
    bad = ~np.isfinite(flat).reshape(-1, 32).all(1)
    calm = flat.copy().reshape(-1, 32)
    calm[bad] = 0
    blocks = oracle.quantize(fmt, calm.reshape(-1, dim)).reshape(-1, BLOCK[fmt])
    d = np.ascontiguousarray(blocks[:, :2]).view(np.float16)[:, 0].copy()
    if fmt == Q8_0:
        q = blocks[:, 2:].view(np.int8).astype(np.int64)
    else:
        q = np.concatenate([blocks[:, 2:] & 15, blocks[:, 2:] >> 4], 1).astype(np.int64) - 8
    bad |= ~np.isfinite(d)
    q[bad | (d == 0)] = 0
    d[bad] = np.nan
    return q.reshape(*shape, dim), d.reshape(*shape, dim // 32)


def values(q, d):
    """f64 [..., D] that codes and scales stand for."""
    return q * np.repeat(d.astype(np.float64), 32, -1)


def place(t):
    s, h, g, i = t // 32, t % 32 // 16, t % 16 // 4, t % 4
    return 16 * g + 8 * s + 4 * h + i


def code_at(fmt, is_values, dim, t, d):
    """(byte, shift) in a group of 64 tokens of the code of token t, dimension d."""
    b = d // 32
    if is_values:
        lane = place(t) // 16 * 16 + d % 16
        p, e = d % 32 // 16, place(t) % 16
        if fmt == Q8_0:
            return b * 2048 + p * 1024 + lane * 16 + e, 0
        nib = e % 8 // 2 + 4 * (e % 2)
        return b * 1024 + lane * 16 + p * 8 + e // 8 * 4 + nib // 2, nib % 2 * 4
    lane, e = d % 32 // 8 * 16 + t % 16, d % 8
    if fmt == Q8_0:
        held, at, shift = dim // 4, 8 * b + e, 0
    else:
        nib = e // 2 + 4 * (e % 2)
        held, at, shift = dim // 8, 4 * b + nib // 2, nib % 2 * 4
    piece = at // 16
    return t // 16 * 64 * held + piece * 1024 + lane * min(16, held - 16 * piece) + at % 16, shift


def scale_at(fmt, dim, t, b):
    return (64 * dim if fmt == Q8_0 else 32 * dim) + 2 * (64 * b + place(t))


_maps = {}


def maps(fmt, is_values, dim):
    key = fmt, is_values, dim
    if key not in _maps:
        at = np.array([[code_at(fmt, is_values, dim, t, d) for d in range(dim)] for t in range(64)])
        sc = np.array([[scale_at(fmt, dim, t, b) for b in range(dim // 32)] for t in range(64)])
        _maps[key] = at[..., 0], at[..., 1], sc
    return _maps[key]


def write(cache, fmt, is_values, page, head, t, q, d):
    """Codes [D] and scales [D / 32] of the token at offset t of a page into cache uint8 [pages, heads, page size, row]."""
    dim = len(q)
    at, shift, sc = maps(fmt, is_values, dim)
    size = 64 * row_bytes(fmt, dim)
    flat = cache[page, head].reshape(-1)[t // 64 * size:][:size]
    at, shift, sc = at[t % 64], shift[t % 64], sc[t % 64]
    if fmt == Q8_0:
        flat[at] = q + 128
    else:
        for half in (0, 4):
            m = shift == half
            flat[at[m]] = (flat[at[m]] & (0xF0 >> half)) | ((q[m] + 8) << half)
    raw = d.view(np.uint8).reshape(-1, 2)
    flat[sc], flat[sc + 1] = raw[:, 0], raw[:, 1]


def write_many(cache, fmt, is_values, pages, tokens, q, d):
    """Whole sequences: q [L, H, D], d [L, H, D / 32], the token of row n at offset tokens[n] of page pages[n]."""
    dim, heads = q.shape[-1], q.shape[1]
    at, shift, sc = maps(fmt, is_values, dim)
    size = 64 * row_bytes(fmt, dim)
    flat = cache.reshape(cache.shape[0], heads, -1)
    p, h = pages[:, None, None], np.arange(heads)[None, :, None]
    base = (tokens // 64 * size)[:, None, None]
    a, sh, c = at[tokens % 64][:, None] + base, np.broadcast_to(shift[tokens % 64][:, None], q.shape), sc[tokens % 64][:, None] + base
    if fmt == Q8_0:
        flat[p, h, a] = q + 128
    else:
        np.bitwise_and.at(flat, (p, h, a), (0xF0 >> sh).astype(np.uint8))
        np.bitwise_or.at(flat, (p, h, a), ((q + 8) << sh).astype(np.uint8))
    raw = np.ascontiguousarray(d).view(np.uint8).reshape(*d.shape, 2)
    flat[p, h, c], flat[p, h, c + 1] = raw[..., 0], raw[..., 1]


class Cache:
    """Sequences of given lengths in pages of a pool, in an order of no meaning; what no token wrote is garbage."""

    def __init__(self, seed, fmt_k, fmt_v, heads, dim, page_size, lengths, k_scale=1.0, v_scale=1.0, spare=1, width=None):
        g = np.random.default_rng(seed)
        self.fmt_k, self.fmt_v, self.heads, self.dim, self.page_size = fmt_k, fmt_v, heads, dim, page_size
        self.lengths = np.array(lengths, dtype=np.int32)
        held = [-(-n // page_size) for n in lengths]
        pages = sum(held) + spare
        width = max(held + [1]) if width is None else width
        self.table = np.full((len(lengths), width), -1, dtype=np.int32)
        order = g.permutation(pages)
        self.k_cache = g.integers(0, 256, (pages, heads, page_size, row_bytes(fmt_k, dim)), dtype=np.uint8)
        self.v_cache = g.integers(0, 256, (pages, heads, page_size, row_bytes(fmt_v, dim)), dtype=np.uint8)
        self.k, self.v = [], []
        used = 0
        for s, n in enumerate(lengths):
            self.table[s, :held[s]] = order[used:used + held[s]]
            used += held[s]
            k = (k_scale * g.standard_normal((n, heads, dim))).astype(np.float32)
            v = (v_scale * g.standard_normal((n, heads, dim))).astype(np.float32)
            self.k.append(k)
            self.v.append(v)
        self.write()

    def places(self, s, n):
        pos = np.arange(n)
        return self.table[s, pos // self.page_size], pos % self.page_size

    def write(self):
        """(Re)writes every sequence from self.k and self.v; self.kq and self.vq: the f64 values they then stand for."""
        self.kq, self.vq = [], []
        for s, n in enumerate(self.lengths):
            for fmt, is_values, cache, x, out in ((self.fmt_k, False, self.k_cache, self.k[s], self.kq),
                                                  (self.fmt_v, True, self.v_cache, self.v[s], self.vq)):
                q, d = quantize(fmt, x)
                if n:
                    write_many(cache, fmt, is_values, *self.places(s, int(n)), q, d)
                out.append(values(q, d))


def attention(q, k, v, positions, scale, causal=True, window=0, softcap=0.0, seen=None):
    """One sequence in 64 bits: q [n, Hq, D], k, v [L, H, D], positions [n]; seen: [L], positions that have a page.
    Returns out [n, Hq, D], lse [n, Hq], A = sum_j p_j |v_j| [n, Hq, D] and E = max_j scale sum_d |q_d k_jd| [n, Hq]
    over the positions that a row sees."""
    n, hq, dim = q.shape
    length, heads = k.shape[:2]
    out, big = np.zeros((n, hq, dim)), np.zeros((n, hq, dim))
    lse, top = np.full((n, hq), -np.inf), np.zeros((n, hq))
    positions = np.asarray(positions)
    j = np.arange(length)
    m = np.ones((n, length), dtype=bool) if seen is None else np.tile(seen, (n, 1))
    if causal:
        m &= j <= positions[:, None]
    if window:
        m &= j > positions[:, None] - window
    rows = m.any(1)
    if not rows.any():
        return out, lse, big, top
    hidden = ~m[rows]
    for h in range(hq):
        kk, vv = k[:, h // (hq // heads)], v[:, h // (hq // heads)]
        with np.errstate(invalid="ignore"):
            s = scale * (q[rows, h] @ np.where(np.isnan(kk), 0.0, kk).T)
            s = np.where(np.isnan(kk).any(1), np.nan, s)
            if softcap:
                s = softcap * np.tanh(s / softcap)
            s[hidden] = -np.inf
            peak = s.max(1, keepdims=True)
            p = np.exp(s - peak)
            lse[rows, h] = peak[:, 0] + np.log(p.sum(1))
            p /= p.sum(1, keepdims=True)
        o, a = p @ np.nan_to_num(vv), p @ np.abs(np.nan_to_num(vv))
        for t, d in np.argwhere(np.isnan(vv)):
            o[~hidden[:, t], d] = np.nan
        out[rows, h], big[rows, h] = o, a
        e = np.abs(q[rows, h]) @ np.abs(np.nan_to_num(kk)).T
        e[hidden] = 0
        top[rows, h] = abs(scale) * e.max(1)
    return out, lse, big, top
