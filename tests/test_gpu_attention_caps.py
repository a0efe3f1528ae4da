"""Soft caps of any size: softcap * tanh(x / softcap) keeps x's relative accuracy
however far the cap lies above the scores, and a cap out of their reach is none."""
import numpy as np
import pytest

import cache_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from attention_bounds import run_close  # noqa: E402
from test_gpu_attention import FMTS  # noqa: E402

# kernel, type, lengths, new tokens, heads of the cache, query heads to each
ROWS = [("rows", t, [40, 300, 3], [1, 5, 3], 2, 3) for t in ("f32", "f16", "bf16")]
MANY = [("many", t, [200, 75, 77], [76, 75, 77], 8, 8) for t in ("f16", "bf16")]


@pytest.mark.parametrize("kernel,dtype,lengths,new,heads,per", ROWS + MANY)
@pytest.mark.parametrize("fk,fv,dim", [("q8", "q8", 64), ("q4", "q8", 128)])
@pytest.mark.parametrize("window", [0, 3])
@pytest.mark.parametrize("cap", [0.5, 3.0, 50.0, 1e3, 1e4, 1e6, 1e8, 2e38])
def test_caps(cap, window, fk, fv, dim, kernel, dtype, lengths, new, heads, per):
    print(f"cap {cap} {window} {fk} {fv} {dim} {kernel} {dtype}", flush=True)
    c = ref.Cache(300, FMTS[fk], FMTS[fv], heads, dim, 64, lengths)
    run_close(kernel, c, dtype, per, new, seed=301, q_scale=2.0, window=window, softcap=cap)


@pytest.mark.parametrize("kernel,dtype,lengths,new,heads,per", ROWS + MANY)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-3])
def test_scales_with_a_cap(scale, kernel, dtype, lengths, new, heads, per):
    c = ref.Cache(310, FMTS["q8"], FMTS["q4"], heads, 64, 64, lengths)
    for cap in (2.0, 1e8):
        run_close(kernel, c, dtype, per, new, seed=311, scale=scale, softcap=cap)


@pytest.mark.parametrize("kernel,dtype,lengths,new,heads,per", ROWS + MANY)
@pytest.mark.parametrize("cap", [3.0, 1e8])
def test_what_is_not_finite_under_a_cap(cap, kernel, dtype, lengths, new, heads, per):
    """A cap does not turn a NaN into a number, nor let a key or value touch a row that does not see it."""
    c = ref.Cache(320, FMTS["q8"], FMTS["q8"], heads, 64, 64, lengths)
    c.v[0][lengths[0] - 1, 0, 40] = np.nan
    c.k[0][lengths[0] - 2, 1, 5] = np.inf
    c.k[1][0, 0, 9] = np.nan
    c.write()
    out, _ = run_close(kernel, c, dtype, per, new, seed=321, window=30, softcap=cap)
    assert torch.isnan(out).any() and not torch.isnan(out).all()
