"""Combines and products with one activation row per slot in row tiles of 64 and 128 rows, and weights past
2^32 bytes, against plain implementations in 64 bits (tolerances as in test_gpu_experts.py).

The tile is the smallest of 32, 64 and, but for f32, 128 rows that leaves one round of 256 workgroups of 256
weight rows, else the largest; the outputs of the f32 products that a combine sums leave the larger ones in
two passes.  The expert's numbers of pairs differ widely, so tiles end in either pass and in every body."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_matmul_gguf_amd as qmm  # noqa: E402

from test_gpu_experts import BAR, FMTS, TYPES, act_ref, acts, close, k_of, product_ref, skewed, weights_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    qmm.lib()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("t,e,k,n,mult", [
    (750, 9, 4, 1290, 2),   # 128 rows (f32: 64)
    (1400, 5, 1, 1300, 1),  # 64 rows
    (500, 9, 4, 1291, 3),   # 64 rows, outputs one by one
    (2100, 3, 2, 516, 1),   # 64 rows
    (3000, 2, 2, 1031, 1),  # 128 rows, two experts of which one has no pairs
])
def test_rows_per_slot_in_large_tiles(fmt, dtype, t, e, k, n, mult):
    print(f"slots {fmt} {dtype} T={t} E={e} k={k} N={n} mult={mult}", flush=True)
    f, kk = FMTS[fmt], k_of(FMTS[fmt], mult)
    b, w, wa = weights_of(f, 400 + t, e * n, kk)
    wd = torch.from_numpy(b.reshape(e, n, -1)).cuda()
    ids_h = skewed(401 + t, t, e, k)
    ids_h[np.random.default_rng(402 + t).random((t, k)) < 0.05] = -1
    ids_h[t // 3] = -1
    h, hh = acts(403 + t, (t, k, kk), TYPES[dtype])
    y, a = product_ref(w, wa, e, n, ids_h, hh)
    ids = torch.from_numpy(ids_h).cuda()
    close(qmm.experts_matmul(f, wd, h, ids), y, BAR * a, "experts_matmul per slot")
    g = np.random.default_rng(404 + t).random((t, k)).astype(np.float32)
    gd = g.astype(np.float64)[:, :, None]
    got = qmm.experts_combine(f, wd, h, ids, torch.from_numpy(g).cuda())
    close(got, (y * gd).sum(1), BAR * (a * gd).sum(1), "experts_combine")
    assert (got[t // 3] == 0).all()


@pytest.mark.parametrize("count", [1, 31, 32, 33, 64, 65, 95, 96, 97, 127, 128, 129, 192, 193])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fmt", ["Q8_0", "Q4_0", "Q4_K"])
def test_a_last_tile_of_any_count(fmt, dtype, count):
    """One expert with `count` pairs beside a large one: what its last tile writes, and nothing beyond."""
    f, e, n, k, t = FMTS[fmt], 3, 1290, 1, 3000
    kk = k_of(f, 1)
    b, w, wa = weights_of(f, 420, e * n, kk)
    wd = torch.from_numpy(b.reshape(e, n, -1)).cuda()
    ids_h = np.full((t, k), 2, np.int32)
    ids_h[np.random.default_rng(421 + count).permutation(t)[:count]] = 1
    h, hh = acts(422, (t, k, kk), TYPES[dtype])
    y, a = product_ref(w, wa, e, n, ids_h, hh)
    close(qmm.experts_combine(f, wd, h, torch.from_numpy(ids_h).cuda(), torch.ones((t, k)).cuda()), y[:, 0], BAR * a[:, 0], "combine")


@pytest.mark.parametrize("t", [1, 30, 100, 1100])
def test_glu_and_combine_past_32_bit_offsets(t):
    """64 x 33000 x 2048 in Q8_0: 4.6e9 bytes; of the last expert the last 40 rows, past 2^32, are not zero."""
    f, e, n, k = qmm.Q8_0, 64, 33000, 2048
    b, w, wa = weights_of(f, 250, 40, k)
    wd = torch.zeros((e, n, b.shape[1]), dtype=torch.uint8, device="cuda")
    wd[-1, -40:] = torch.from_numpy(b).cuda()
    x, xh = acts(251, (t, k), torch.float16)
    ids = torch.full((t, 1), e - 1, dtype=torch.int32).cuda()
    y, a = xh @ w.T, np.abs(xh) @ wa.T
    for act in ("silu", "gelu"):
        h = qmm.experts_glu(f, wd, wd, x, ids, act=act)[:, 0]
        ag = act_ref(y, act)
        slack = 1.13 * BAR * a * (np.abs(y) + BAR * a) + np.abs(y) * BAR * a + 2.0**-20 * np.abs(ag * y)
        close(h[:, -40:], ag * y, slack, act)
        assert (h[:, :-40] == 0).all()
    got = qmm.experts_combine(f, wd, x[:, None].contiguous(), ids, torch.full((t, 1), 0.75).cuda())
    close(got[:, -40:], 0.75 * y, 0.75 * BAR * a, "combine")
    assert (got[:, :-40] == 0).all()
