"""Values at the ends of their ranges against plain implementations in 64 bits.

Tolerances are those of test_gpu_experts.py: 1e-5 of the sum of magnitudes for f32 sums, one rounding to
the output's type, and what the header states that activations and scales lose on the way in.
"""
import numpy as np
import pytest

import oracle
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_matmul_gguf_amd as qmm  # noqa: E402

from test_gpu_experts import BAR, FMTS, TYPES, close, f64, route_ref, w4_case, weights_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    qmm.lib()


def w4_scaled(seed, n, k, group, sdtype, low, high):
    """4-bit weights whose scales' magnitudes are spread over 2^low .. 2^high, the last group at the top."""
    q, s, z, _ = w4_case(seed, n, k, group, True, sdtype)
    g = np.random.default_rng(seed + 1)
    mag = np.exp2(g.uniform(low, high, s.shape))
    mag[:, -1] = 2.0**high
    s = torch.from_numpy((mag * np.where(g.random(s.shape) < 0.5, -1, 1)).astype(np.float32)).to(sdtype)
    qh = q.cpu().numpy()
    codes = np.stack([qh & 15, qh >> 4], -1).reshape(n, k).astype(np.float64) - np.repeat(f64(z), group, 1)
    return q, s.cuda(), z, codes, np.repeat(f64(s), group, 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sdtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("m", [1, 60, 1500])
@pytest.mark.parametrize("size,low,high", [
    (1e-6, 90, 106.3), (1e-30, 60, 127.9), (1.0, 80, 112), (2.0**-126, 20, 127.9), (1e25, -100, -80), (1e32, -130, -90),
    (1.0, -149, -100), (2.0**100, -60, -20),
])
def test_w4_scales_of_any_size(dtype, sdtype, group, m, size, low, high):
    """Finite results where scale times activation is finite, however large or small either is.  Scales
    enter to 2^-24 of themselves or 2^-107, sums to 2^-121 of the row's largest per 32 values."""
    print(f"w4 {dtype} M={m} G={group} {sdtype} x {size} scales 2^{low}..2^{high}", flush=True)
    n, k = 1030, 256
    q, s, z, codes, scale = w4_scaled(300, n, k, group, TYPES[sdtype], low, high)
    x = torch.from_numpy((synth.acts_f32(301, m, k).astype(np.float64) * size).astype(np.float32)).to(TYPES[dtype])
    xh = x.double().numpy()
    a = np.abs(xh) @ np.abs(codes * scale).T
    lost = np.maximum(2.0**-24 * np.abs(scale), 2.0**-107) * np.abs(codes)
    top = np.abs(xh).max(1, keepdims=True)
    slack = BAR * a + np.abs(xh) @ lost.T + k / 32 * 2.0**-121 * top
    slack += np.maximum(2.0**-39 * top, 2.0**-151) * np.abs(codes * scale).sum(1)  # the activations'
    y = qmm.w4_matmul(q, s, x.cuda(), zeros=z)
    assert torch.isfinite(y).all()
    close(y, xh @ (codes * scale).T, slack, "w4")


@pytest.mark.parametrize("m", [1, 60, 1500])
def test_w4_largest_scales_in_long_rows(m):
    """K = 33024 with every product of one sign, zero points of 255: the largest sums there are."""
    n, k, group = 37, 33024, 128
    g = np.random.default_rng(310)
    q = torch.zeros((n, k // 2), dtype=torch.uint8).cuda()
    z = torch.full((n, k // group), 255, dtype=torch.uint8).cuda()
    s = torch.full((n, k // group), 3.0e38, dtype=torch.float32).cuda()
    x = torch.from_numpy((2.0**-20 * (1 + g.random((m, k)))).astype(np.float32))
    y = qmm.w4_matmul(q, s, x.cuda(), zeros=z)
    want = -(f64(x).sum(1, keepdims=True) * 255.0 * f64(s)[0, 0]) * np.ones((1, n))
    assert (np.abs(want) > 3.5e38).all() and (y == -torch.inf).all()  # too large for the type: infinite, not NaN
    small = x * 2.0**-10
    want = -(f64(small).sum(1, keepdims=True) * 255.0 * f64(s)[0, 0]) * np.ones((1, n))
    assert (np.abs(want) < 3.0e38).all()
    close(qmm.w4_matmul(q, s, small.cuda(), zeros=z), want, (k / 32 + 64) * 2.0**-24 * np.abs(want), "long rows")


def few_values(dtype, m, k, at, outlier, values):
    """Rows that are zero but for an outlier at `at` and values[i % len] at element 7."""
    x = torch.zeros((m, k), dtype=torch.float64)
    x[:, at] = outlier
    x[:, 7] = torch.tensor([values[i % len(values)] for i in range(m)], dtype=torch.float64)
    t = x.to(TYPES[dtype])
    assert torch.equal(t.double(), x)
    return t.cuda(), x.numpy()


def hollow(fmt, seed, n, k, at):
    """Blocks of weights up to about 2^16 in which element `at` of every row is exactly zero."""
    w = synth.weights_f32(seed, n, k) * np.float32(2.0**19)
    w[:, at] = 0
    b = oracle.quantize(fmt, w)
    if fmt == qmm.Q4_K:  # without minima, and the code itself zero
        b = b.reshape(n, -1, 144).copy()
        b[:, :, 2:4] = 0
        sub, i = at % 256 // 32, at % 32
        b[:, at // 256, 16 + sub // 2 * 32 + i] &= 0x0F if sub % 2 else 0xF0
        b = b.reshape(n, -1)
    v = oracle.dequantize(fmt, b, k)
    assert (v[:, at] == 0).all() and (v[:, 7] != 0).any()
    return b, v


def product(fmt, b, n, x, how):
    """x . W^T through experts_matmul, or (combine) through experts_combine with weight 1."""
    wd = torch.from_numpy(b.reshape(1, n, -1)).cuda()
    ids = torch.zeros((len(x), 1), dtype=torch.int32).cuda()
    if how == "combine":
        return qmm.experts_combine(fmt, wd, x[:, None].contiguous(), ids, torch.ones((len(x), 1)).cuda())
    return qmm.experts_matmul(fmt, wd, x, ids)[:, 0]


SMALL = {
    # what is lost of element 7 beside an outlier: nothing of an f16 value, else 2^-22 of it or 2^-39 of the outlier
    "f16": [(60000.0, [2.0**-24, 3 * 2.0**-24, 5 * 2.0**-24, 1023 * 2.0**-24, 2.0**-14, 2047 * 2.0**-13]),
            (65504.0, [2.0**-24, 7 * 2.0**-24]), (32768.0, [2.0**-24, 1025 * 2.0**-23]), (2.0**-14, [2.0**-24, 3 * 2.0**-24])],
    "bf16": [(1.0, [2.0**-39, 2.0**-38, 255 * 2.0**-46, 129 * 2.0**-40, 171 * 2.0**-30]), (2.0**100, [2.0**61, 2.0**62, 2.0**70]),
             (2.0**-110, [2.0**-126, 2.0**-130, 2.0**-133])],
    "f32": [(1.0, [2.0**-39, 2.0**-38, 255 * 2.0**-46, 16777215 * 2.0**-50, 2.0**-20 + 2.0**-43]), (2.0**100, [2.0**61, 2.0**62 + 2.0**40]),
            (1.9999998807907104, [2.0**-38, 3 * 2.0**-40]), (2.0**-115, [2.0**-126, 2.0**-140, 2.0**-149])],
}


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fmt,how", [(f, h) for f in FMTS for h in ("run", "combine")] + [("W4", "run")])
@pytest.mark.parametrize("m", [1, 60, 1500])
def test_a_small_value_beside_an_outlier_of_weight_zero(fmt, dtype, m, how):
    """Each value by itself: f16 activations enter as they are, others to 2^-22 of themselves, 2^-39 of
    their row's largest or 2^-151."""
    k, n, at = 256, 1030 if how == "run" else 40, 100
    if fmt == "W4":
        q, s, z, _ = w4_case(320, n, k, 64, False, torch.float32)
        s = s * 2.0**20
        q[:, 50] = 0x88
        qh = q.cpu().numpy()
        w = (np.stack([qh & 15, qh >> 4], -1).reshape(n, k).astype(np.float64) - 8) * np.repeat(f64(s), 64, 1)
    else:
        b, w = hollow(FMTS[fmt], 321, n, k, at)
    for outlier, values in SMALL[dtype]:
        x, xh = few_values(dtype, m, k, at, outlier, values)
        y = qmm.w4_matmul(q, s, x) if fmt == "W4" else product(FMTS[fmt], b, n, x, how)
        v = np.abs(xh[:, 7:8])
        lost = 0 * v if dtype == "f16" else np.maximum(np.maximum(2.0**-22 * v, 2.0**-39 * outlier), 2.0**-151)
        close(y, xh[:, 7:8] * w[None, :, 7], (lost + BAR * v) * np.abs(w[None, :, 7]), f"{outlier} {values}")


@pytest.mark.parametrize("fmt", list(FMTS) + ["W4"])
@pytest.mark.parametrize("m", [1, 60, 1500])
def test_rows_of_the_largest_half(fmt, m):
    """Rows of 65504 throughout, of either sign, in every sub-block sum the largest there is."""
    k, n = 512, 1030
    x = torch.full((m, k), 65504.0, dtype=torch.float16)
    x[1::3] *= -1
    x[2::3, ::2] *= -1
    xh = x.double().numpy()
    if fmt == "W4":
        q, s, z, _ = w4_case(330, n, k, 64, True, torch.float16)
        s, qh = s.float() * 2.0**-10, q.cpu().numpy()
        codes = np.stack([qh & 15, qh >> 4], -1).reshape(n, k).astype(np.float64) - np.repeat(f64(z), 64, 1)
        w = codes * np.repeat(f64(s), 64, 1)
        y, wa = qmm.w4_matmul(q, s, x.cuda(), zeros=z), np.abs(w)
    else:
        b, w, wa = weights_of(FMTS[fmt], 331, n, k)
        y = product(FMTS[fmt], b, n, x.cuda(), "run")
    want, a = xh @ w.T, np.abs(xh) @ wa.T
    fits = np.abs(want) + BAR * a < 65504
    assert fits.any()
    got = f64(y)
    assert np.isfinite(got[fits]).all()
    assert (np.abs(got - want) <= BAR * a + 2.0**-11 * (np.abs(want) + BAR * a) + 2.0**-25)[fits].all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t,e,k,groups,tg,gt", [
    (1, 8, 3, 1, 1, 1), (9, 64, 64, 1, 1, 1), (33, 160, 6, 8, 3, 2), (5, 96, 20, 32, 5, 1), (4, 1024, 64, 64, 10, 2), (3, 7, 7, 7, 3, 2),
])
def test_route_with_biases_that_are_not_finite(dtype, score, renorm, t, e, k, groups, tg, gt):
    """A bias of -inf or NaN takes its expert out of the choice and out of its group's score; one of +inf
    puts it first.  The scores, softmax's sum among them, are of the logits alone."""
    print(f"route {dtype} {score} renorm={renorm} T={t} E={e} k={k} groups={groups}/{tg}/{gt}", flush=True)
    g = np.random.default_rng(340 + e)
    l = g.standard_normal((t, e)) * 2
    l[:, 3] = 9.0  # most of the weight, and out of the choice
    l[-1, 1::3] = -np.inf
    x = torch.from_numpy(l.astype(np.float32)).to(TYPES[dtype])
    b = (0.1 * g.standard_normal(e)).astype(np.float32)
    b[g.random(e) < 0.2] = -np.inf
    b[g.random(e) < 0.1] = np.nan
    b[3] = -np.inf
    b[5] = np.inf
    if groups > 1:
        b[:e // groups] = np.nan  # a group of which nothing is left
    for bias in (b, np.full(e, -np.inf, np.float32), np.full(e, np.nan, np.float32)):
        ids, w = qmm.route_experts(x.cuda(), k, score, torch.from_numpy(bias).cuda(), groups, tg, gt, renorm, 1.5)
        ri, rw = route_ref(x.double().numpy(), k, score, bias, groups, tg, gt, renorm, 1.5)
        assert np.array_equal(ids.cpu().numpy(), ri)
        assert np.all(np.abs(f64(w) - rw) <= 2.0**-24 * (1 + 2.0**-20) * np.abs(rw) + 2.0**-150)
        if not np.isfinite(bias).any():
            assert (ids == -1).all() and (w == 0).all()
