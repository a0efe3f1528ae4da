"""The bounds that attention is held to tell its arithmetic from one that loses
bits: numpy does what a kernel does, and with a part left out it passes them no
more."""
import numpy as np
import pytest

import cache_ref as ref
from attention_bounds import BF16, F16, bounds
from exact_values import cancelling
from test_gpu_attention import check, largest

torch = pytest.importorskip("torch")


def half(x):
    return x.astype(np.float16).astype(np.float64)


def attention(c, q, window, keys_rounded, probabilities_rounded, values_rounded):
    """One sequence as a kernel has it: out, lse."""
    k, v, n, m = c.kq[0], c.vq[0], int(c.lengths[0]), len(q)
    pos, j = np.arange(n - m, n)[:, None], np.arange(n)[None]
    seen = (j <= pos) & (j > pos - window if window else True)
    out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    per = q.shape[1] // c.heads
    for h in range(q.shape[1]):
        kk, vv = k[:, h // per], v[:, h // per]
        s = np.where(seen, c.dim ** -0.5 * q[:, h] @ (half(kk) if keys_rounded else kk).T, -np.inf)
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        total = p.sum(1, keepdims=True)
        p = half(64 * p) / 64 if probabilities_rounded else p
        out[:, h] = p @ (half(vv) if values_rounded else vv) / total
        lse[:, h] = (top + np.log(total))[:, 0]
    return out, lse


def held(kernel, dt, c, q, window, got, exact_values):
    """Whether (out, lse) pass the bounds, each for itself."""
    n, m = int(c.lengths[0]), len(q)
    o, l, big, top = ref.attention(q, c.kq[0], c.vq[0], np.arange(n - m, n), c.dim ** -0.5, True, window)
    tol, of_lse = bounds(kernel, dt, c.dim, window or n, big, top, largest(c.vq[0]), l, exact_values=exact_values)
    result = []
    for g, w, t in ((torch.from_numpy(got[0]).to(dt), o, tol), (torch.from_numpy(got[1]).float(), l, of_lse)):
        try:
            check(g, w, t, "")
            result.append(True)
        except AssertionError:
            result.append(False)
    return tuple(result)


@pytest.mark.parametrize("fk,fv", [(8, 8), (2, 2), (8, 2), (2, 8)])
@pytest.mark.parametrize("dim", [64, 128])
def test_parts(dim, fk, fv):
    c = cancelling(330, fk, fv, 2, dim, 64, [200])
    rng = np.random.default_rng(331)
    for scale, window in ((1.0, 1), (0.05, 4)):
        q = half(rng.standard_normal((75, 6, dim)) * scale)
        assert held("many", F16, c, q, window, attention(c, q, window, False, False, True), True) == (True, True)
        assert held("rows", F16, c, q, window, attention(c, q, window, False, True, False), True) == (True, True)
        assert held("rows", BF16, c, q, window, attention(c, q, window, False, True, False), True) == (True, True)
        assert held("many", BF16, c, q, window, attention(c, q, window, True, True, True), True) == (True, True)
        if window == 1:  # lse is the score: keys that have lost bits
            assert not held("many", F16, c, q, window, attention(c, q, window, True, False, True), True)[1]
            assert not held("rows", F16, c, q, window, attention(c, q, window, True, True, False), True)[1]
            assert not held("rows", BF16, c, q, window, attention(c, q, window, True, True, False), True)[1]
        else:  # probabilities that have
            assert not held("many", F16, c, q, window, attention(c, q, window, False, True, True), True)[0]
