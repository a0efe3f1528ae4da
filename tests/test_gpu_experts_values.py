"""Values at the ends of their ranges against plain implementations in 64 bits.

Tolerances are those of test_gpu_experts.py: 1e-5 of the sum of magnitudes for f32 sums, one rounding to
the output's type, and what the header states that activations and scales lose on the way in.
"""
import numpy as np
import pytest

import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_matmul_gguf_amd as qmm  # noqa: E402

from test_gpu_experts import BAR, TYPES, close, f64, w4_case  # noqa: E402


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
