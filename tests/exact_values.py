"""Caches whose values f16 holds as they are, and whose tokens cancel four by four:
under nearly equal probabilities outputs are small against sum p |v|, so that the
rounding of outputs hides little of what the probabilities lost."""
import numpy as np

import cache_ref as ref


def cancelling(seed, fmt_k, fmt_v, heads, dim, page_size, lengths, **kw):
    """A `cache_ref.Cache` with values code * 2^-7 (Q8_0, codes to 127) or 2^-3 (Q4_0, to 8), the largest in every
    block, and signs + + - - from token to token."""
    c = ref.Cache(seed, fmt_k, fmt_v, heads, dim, page_size, lengths, **kw)
    g = np.random.default_rng(seed + 1)
    top, step = (127, 2.0**-7) if fmt_v == ref.Q8_0 else (8, 2.0**-3)
    code = g.integers(1, top, (heads, dim // 32, 32))
    code[..., 0] = top
    base = (g.permuted(code, axis=-1) * g.choice([-1, 1], code.shape)).reshape(heads, dim) * step
    for s, n in enumerate(lengths):
        sign = np.where(np.arange(n) % 4 < 2, 1.0, -1.0)
        c.v[s] = (sign[:, None, None] * base).astype(np.float32)
    c.write()
    for s in range(len(lengths)):
        assert np.array_equal(c.vq[s], c.v[s]) and np.array_equal(c.vq[s].astype(np.float16), c.v[s])
    return c
