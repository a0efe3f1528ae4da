"""Attention held to each kernel's own bounds: scores by lse under a window of one
position, probabilities by values that f16 holds and that cancel, and batches of
more than 64 sequences with either kernel, in one piece and in several."""
import numpy as np
import pytest

import cache_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_matmul_gguf_amd as qmm  # noqa: E402
from attention_bounds import bounds, run_close  # noqa: E402
from exact_values import cancelling  # noqa: E402
from test_gpu_attention import FMTS, check, gpu, largest, starts_of  # noqa: E402

CODES = {"f32": qmm.F32, "f16": qmm.F16, "bf16": qmm.BF16}
FORMATS = [("q8", "q8"), ("q4", "q4"), ("q8", "q4"), ("q4", "q8")]
# kernel, type, lengths, new tokens, heads of the cache, query heads to each: 16 rows at a time; 608 on average
ROWS = [("rows", t, [200, 3, 64], [75, 3, 1], 2, 3) for t in CODES]
MANY = [("many", t, [200, 75, 77], [76, 75, 77], 8, 8) for t in ("f16", "bf16")]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    qmm.lib()


@pytest.mark.parametrize("kernel,dtype,lengths,new,heads,per", ROWS + MANY)
@pytest.mark.parametrize("fk,fv", FORMATS)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_scores_and_probabilities(dim, fk, fv, kernel, dtype, lengths, new, heads, per):
    if kernel == "many" and dtype == "f16" and dim == 256:
        kernel = "rows"  # (the parts of f16 rows do not fit)
    print(f"close {kernel} {dtype} {fk} {fv} {dim}", flush=True)
    c = cancelling(340 + dim, FMTS[fk], FMTS[fv], heads, dim, 64, lengths)
    run_close(kernel, c, dtype, per, new, seed=341, window=1, exact_values=True)
    run_close(kernel, c, dtype, per, new, seed=342, window=4, q_scale=0.05, exact_values=True)
    run_close(kernel, c, dtype, per, new, seed=343, exact_values=True)


def batch(seed, count, new, lengths):
    """count sequences with new and old tokens in the given ranges, some of them with no rows, one of no tokens."""
    g = np.random.default_rng(seed)
    m = g.integers(*new, count)
    n = np.maximum(m, g.integers(*lengths, count))
    m[3::17] = 0
    n[3], n[-1] = 0, lengths[1]
    return [int(x) for x in n], [int(x) for x in m]


# kernel, types, sequences, new tokens, tokens, query heads, whether in pieces
@pytest.mark.parametrize("kernel,dtype,count,new,lengths,per,cut", [
    (k, t, *rest) for k, types, *rest in [
        ("many", ("f16", "bf16"), 65, (115, 131), (131, 500), 2, False),
        ("many", ("f16", "bf16"), 65, (115, 131), (600, 1400), 2, True),
        ("many", ("f16", "bf16"), 100, (64, 71), (530, 700), 4, True),
        ("rows", ("f32", "f16", "bf16"), 65, (1, 4), (500, 2600), 4, True),
        ("rows", ("f32", "f16", "bf16"), 120, (1, 6), (500, 1100), 3, True),
    ] for t in types], ids=str)
@pytest.mark.parametrize("fk,fv,dim", [("q8", "q4", 64), ("q4", "q8", 128)])
@pytest.mark.parametrize("kw", [dict(), dict(window=100), dict(causal=False)], ids=str)
def test_more_than_64_sequences(kw, fk, fv, dim, kernel, dtype, count, new, lengths, per, cut):
    print(f"many sequences {kernel} {dtype} {count} {new} {lengths} {per} {fk} {fv} {dim} {kw}", flush=True)
    n, m = batch(count, count, new, lengths)
    c = ref.Cache(350, FMTS[fk], FMTS[fv], 1, dim, 64, n)
    shape = qmm.CacheStruct(c.fmt_k, c.fmt_v, len(c.k_cache), 64, 1, dim, None, None, count, c.table.shape[1], None, None, None)
    if not kw:
        assert (qmm.lib().qmatmul_cache_attention_workspace_bytes(shape, sum(m), per, CODES[dtype], 1, 0, 0) > 0) == cut
    a = run_close(kernel, c, dtype, per, m, seed=351, **kw)
    b = run_close(kernel, c, dtype, per, m, seed=351, **kw)
    assert torch.equal(a[0].nan_to_num(7), b[0].nan_to_num(7)) and torch.equal(a[1].nan_to_num(7), b[1].nan_to_num(7))


@pytest.mark.parametrize("kernel,dtype,lengths,new,heads,per", ROWS + MANY)
@pytest.mark.parametrize("fk,fv", FORMATS)
@pytest.mark.parametrize("low", [10.0, 16.0, 22.0])
def test_small_probabilities_of_large_values(low, fk, fv, kernel, dtype, lengths, new, heads, per):
    """Each row sees a token of value 0 and one of a large value whose probability is e^-low: what is left of it where
    f16 ends, 2^-37 of the value in the rows kernel and 2^-30 in the one for many rows."""
    dim = 64
    c = ref.Cache(360, FMTS[fk], FMTS[fv], heads, dim, 64, lengths)
    g = np.random.default_rng(361)
    for s, n in enumerate(lengths):
        large = (np.arange(n) % 2 == 1)[:, None, None]
        c.k[s] = np.broadcast_to(np.where(large, -low * dim ** -0.5, 0.0), (n, heads, dim)).astype(np.float32)
        c.v[s] = np.where(large, g.uniform(1e4, 4e4, (n, heads, dim)), 0.0).astype(np.float32)
    c.write()
    dt, st = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype], starts_of(new)
    q = torch.ones((int(st[-1]), heads * per, dim), dtype=dt)
    out = qmm.cache_attention(c.fmt_k, c.fmt_v, gpu(c.k_cache), gpu(c.v_cache), q.cuda(), gpu(c.table), gpu(st), gpu(c.lengths), window=2)
    for s, n in enumerate(lengths):
        rows, m = slice(st[s], st[s + 1]), new[s]
        o, l, big, top = ref.attention(q[rows].double().numpy(), c.kq[s], c.vq[s], np.arange(n - m, n), dim ** -0.5, window=2)
        check(out[rows], o, bounds(kernel, dt, dim, 2, big, top, largest(c.vq[s]), l)[0], f"out of sequence {s}")
