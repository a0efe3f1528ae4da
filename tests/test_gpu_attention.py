"""Attention over the quantized paged cache on the GPU, against 64 bits on the
values that the cache's blocks stand for.

Tolerance, with A = sum_j p_j |v_j| and E = the largest scale * sum_d |q_d k_jd|
of the positions that a row sees:
  * a score is off by at most E (u + (D + 8) 2^-24): u is what q or the key
    loses on its way to the matrix cores (f32: two f16 parts, 2^-21 of the row's
    largest value, at most 2^-21 max|q| / |q| more in E than relative to it, so
    2^-19; f16: 0; bf16: keys rounded to f16, 2^-11), the rest D products and
    their scales in f32; the exponent's argument is formed in f32 from the
    score and the running maximum: 2^-22 (E + 4).  exp2 itself: 2^-22;
  * softcap: |tanh'| <= 1, tanh in f32: 2^-21 of the cap;
  * a probability's relative error is twice the score's (the sum of them has it
    too), and the output's error that times A;
  * a probability is rounded to f16, 2^-11, and so is a value (a code times its
    scale) where many rows share it, 2^-11; f32: the code is exact, the
    probability times the scale in two parts, 2^-21;
  * that operand is P d 2^-E in f16, E such that the largest scale d met is
    below 2^(E + 14) and at least 2^(E + 13): below 2^-14 it is off by up to half
    f16's smallest step, 2^-25, which times a code (at most 128) and 2^E is at
    most 2^-38 128 d, or 2^-37 of the largest |v| of the sequence (a block has a
    code of 127 or 8 at least).  Each position can be off by that, and the
    probabilities' sum that divides it is at least 1: L 2^-37 max|v|;
  * sums over L positions in f32: at most L / 16 + 16 roundings of partial sums
    (sixteen or more products enter an accumulator at once), 2^-24 each;
  * one rounding to the output's type.
"""
import math

import numpy as np
import pytest

import cache_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_matmul_gguf_amd as qmm  # noqa: E402

FMTS = {"q8": qmm.Q8_0, "q4": qmm.Q4_0}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {torch.float32: 2.0**-140, torch.float16: 2.0**-24, torch.bfloat16: 2.0**-130}
LOSS_S = {torch.float32: 2.0**-19, torch.float16: 0.0, torch.bfloat16: 2.0**-11}
LOSS_P = {torch.float32: 2.0**-21, torch.float16: 2.0**-10, torch.bfloat16: 2.0**-10}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    qmm.lib()


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def starts_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def largest(v):
    return float(np.nan_to_num(np.abs(v)).max(initial=0.0))


def slack(dt, dim, length, big, top, most, softcap=0.0):
    s = top * (LOSS_S[dt] + (dim + 8) * 2.0**-24) + 2.0**-22 * (top + 4) + 2.0**-22 + softcap * 2.0**-21
    return big * (2 * np.expm1(2 * s)[..., None] / 2 + LOSS_P[dt] + (length / 16 + 16) * 2.0**-24) + length * 2.0**-37 * most, s


def check(got, want, tol, what):
    dt = got.dtype
    g = got.detach().cpu().double().numpy()
    tol = tol + torch.finfo(dt).eps / 2 * (np.abs(want) + tol) + TINY[dt]
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(g - want) <= tol) | (g == want) | (np.isnan(g) & np.isnan(want)))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {g[i]!r} want {want[i]!r} tol {tol[i]!r}")


def run_case(seed, fk, fv, dtype, heads, per, dim, page, lengths, new, causal=True, window=0, softcap=0.0, scale=None,
             q_scale=1.0, v_scale=1.0, max_length=0, cache=None, q=None):
    dt = TYPES[dtype]
    c = cache or ref.Cache(seed, FMTS[fk], FMTS[fv], heads, dim, page, lengths, v_scale=v_scale)
    t = sum(new)
    st = starts_of(new)
    if q is None:
        q = torch.from_numpy((q_scale * np.random.default_rng(seed + 1).standard_normal((t, heads * per, dim))).astype(np.float32))
        q = q.to(dt).cuda()
    lse = torch.empty((t, heads * per), dtype=torch.float32, device="cuda")
    out = qmm.cache_attention(c.fmt_k, c.fmt_v, gpu(c.k_cache), gpu(c.v_cache), q, gpu(c.table), gpu(st), gpu(c.lengths),
                              scale=scale, causal=causal, window=window, softcap=softcap, max_length=max_length, lse=lse)
    qh = q.cpu().double().numpy()
    for s, n in enumerate(lengths):
        rows = slice(st[s], st[s + 1])
        pos = np.arange(n - new[s], n)
        o, l, big, top = ref.attention(qh[rows], c.kq[s], c.vq[s], pos, dim ** -0.5 if scale is None else scale, causal, window, softcap)
        tol, e = slack(dt, dim, n, big, top, largest(c.vq[s]), softcap)
        check(out[rows], o, tol, f"out of sequence {s}")
        check(lse[rows], l, np.where(np.isfinite(l), 2 * e + (n / 16 + 16) * 2.0**-24 + LOSS_P[dt], 0.0), f"lse of sequence {s}")
    return out, lse


# lengths, new tokens, heads of the cache, query heads to each, page size
BATCHES = [
    ([1], [1], 1, 1, 64), ([307], [1], 3, 3, 64), ([64], [1], 1, 8, 64), ([65, 63, 130, 2], [1, 1, 1, 1], 2, 4, 64),
    ([700, 90, 1500], [1, 1, 1], 2, 6, 128), ([40], [40], 2, 3, 64), ([200, 31], [17, 31], 1, 2, 192),
    ([130, 1, 257, 90], [130, 1, 5, 0], 2, 1, 64), ([900], [100], 1, 4, 256), ([333], [333], 1, 1, 64),
    ([600, 700], [5, 3], 1, 16, 64), ([150], [150], 1, 12, 128),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fk,fv", [("q8", "q8"), ("q4", "q4"), ("q8", "q4"), ("q4", "q8")])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("lengths,new,heads,per,page", BATCHES)
def test_attention(lengths, new, heads, per, page, dim, fk, fv, dtype):
    print(f"attention {lengths} {new} {heads}x{per} {dim} {page} {fk} {fv} {dtype}", flush=True)
    run_case(20 + dim, fk, fv, dtype, heads, per, dim, page, lengths, new)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fk,fv,dim", [("q8", "q8", 64), ("q8", "q4", 128), ("q4", "q4", 256), ("q4", "q8", 96)])
@pytest.mark.parametrize("kw", [dict(window=1), dict(window=64), dict(window=100), dict(softcap=20.0, q_scale=8.0),
                                dict(softcap=5.0, window=33), dict(causal=False), dict(scale=0.3), dict(scale=0.0),
                                dict(scale=-0.1)], ids=str)
@pytest.mark.parametrize("lengths,new", [([260, 70], [1, 1]), ([300, 129], [140, 129])])
def test_masks_and_scores(lengths, new, kw, fk, fv, dim, dtype):
    print(f"masks {lengths} {new} {kw} {fk} {fv} {dim} {dtype}", flush=True)
    run_case(30, fk, fv, dtype, 2, 3, dim, 64, lengths, new, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fk,fv,dim", [("q8", "q8", 128), ("q4", "q4", 64)])
@pytest.mark.parametrize("new", [1, 3])
@pytest.mark.parametrize("length", [5000, 20001])
def test_long_sequences_are_split(length, new, fk, fv, dim, dtype):
    a = run_case(40, fk, fv, dtype, 1, 2, dim, 128, [length, 700], [new, 1])
    # a bound on the lengths changes how the work is split; one that is too low does not change the result
    for bound in (length, 256):
        run_case(40, fk, fv, dtype, 1, 2, dim, 128, [length, 700], [new, 1], max_length=bound)
    b = run_case(40, fk, fv, dtype, 1, 2, dim, 128, [length, 700], [new, 1])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # and a call repeats itself bit by bit


def test_rows_that_see_nothing():
    """No tokens, positions before the sequence, tables without pages: zeros and -inf; rows of no sequence stay."""
    heads, dim = 2, 64
    c = ref.Cache(50, 8, 8, heads, dim, 64, [0, 10, 100, 130])
    c.table[3, 0] = 99  # no such page: positions 0..63 of the last sequence are not there
    new = [2, 14, 3, 100]
    st = 3 + starts_of(new)
    t = int(st[-1]) + 5
    for dt in TYPES.values():
        q = torch.randn((t, 2 * heads, dim), device="cuda").to(dt)
        out = torch.full((t, 2 * heads, dim), 7.0, device="cuda", dtype=dt)
        lse = torch.full((t, 2 * heads), 7.0, device="cuda")
        qmm.cache_attention(8, 8, gpu(c.k_cache), gpu(c.v_cache), q, gpu(c.table), gpu(st), gpu(c.lengths), out=out, lse=lse)
        for rows in (slice(0, 3), slice(int(st[-1]), t)):
            assert (out[rows] == 7).all() and (lse[rows] == 7).all()
        qh = q.cpu().double().numpy()
        for s, n in enumerate(c.lengths):
            rows = slice(st[s], st[s + 1])
            seen = np.arange(n) >= 64 if s == 3 else None
            o, l, big, top = ref.attention(qh[rows], c.kq[s], c.vq[s], np.arange(n - new[s], n), dim ** -0.5, seen=seen)
            tol, e = slack(dt, dim, n, big, top, largest(c.vq[s]))
            check(out[rows], o, tol, f"out of sequence {s}")
            check(lse[rows], l, np.where(np.isfinite(l), 2 * e + 2.0**-19 + LOSS_P[dt], 0.0), f"lse of sequence {s}")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fk,fv", [("q8", "q8"), ("q4", "q4")])
@pytest.mark.parametrize("new,per", [(40, 1), (40, 8), (3, 1)])
def test_values_that_are_not_finite(new, per, fk, fv, dtype):
    """A NaN in a key or value reaches the rows that see it (a value: the dimensions of its block) and no others."""
    n, heads, dim = 200, 1, 64
    c = ref.Cache(60, FMTS[fk], FMTS[fv], heads, dim, 64, [n])
    c.v[0][n - 2, 0, 40] = np.nan
    c.v[0][10, 0, 3] = np.inf
    c.write()
    run_case(60, fk, fv, dtype, heads, per, dim, 64, [n], [new], cache=c, window=150)
    c.k[0][n - 1, 0, 5] = np.inf
    c.write()
    run_case(60, fk, fv, dtype, heads, per, dim, 64, [n], [new], cache=c, window=150)
    # and in q: that row alone
    q = torch.randn((new, heads * per, dim), device="cuda").to(TYPES[dtype])
    q[0, 0, 7] = float("nan")
    q[1, 0, 9] = float("inf")
    c = ref.Cache(61, FMTS[fk], FMTS[fv], heads, dim, 64, [n])
    st = gpu(np.array([0, new], np.int32))
    out = qmm.cache_attention(c.fmt_k, c.fmt_v, gpu(c.k_cache), gpu(c.v_cache), q, gpu(c.table), st, gpu(c.lengths))
    bad = torch.isnan(out).any(2)
    assert bad[0, 0] and bad[1, 0] and int(bad.sum()) == 2 and torch.isnan(out[:2, 0]).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fk,fv", [("q8", "q8"), ("q4", "q4"), ("q8", "q4")])
@pytest.mark.parametrize("new,per", [(1, 4), (70, 2)])
def test_the_ends_of_the_range(new, per, fk, fv, dtype):
    """Values far from one: small and large scales beside each other, and all of them small or large."""
    n, dim = 300, 64
    for v_scale, q_scale, mixed in ((1e-3, 1.0, False), (6e3, 1.0, False), (1.0, 1e-3, False), (1.0, 30.0, False), (1.0, 1.0, True)):
        c = ref.Cache(70, FMTS[fk], FMTS[fv], 1, dim, 64, [n], v_scale=v_scale)
        if mixed:
            c.v[0] *= np.exp2(np.random.default_rng(5).integers(-8, 9, (n, 1, 1))).astype(np.float32)
            c.k[0] *= np.exp2(np.random.default_rng(6).integers(-6, 3, (n, 1, 1))).astype(np.float32)
            c.write()
        run_case(71, fk, fv, dtype, 1, per, dim, 64, [n], [new], cache=c, q_scale=q_scale)


def test_strided_queries_and_given_outputs():
    heads, per, dim, n = 2, 3, 128, 50
    c = ref.Cache(80, 8, 8, heads, dim, 64, [n])
    fused = torch.randn((n, heads * (per + 2), dim), device="cuda", dtype=torch.float16)
    args = 8, 8, gpu(c.k_cache), gpu(c.v_cache)
    batch = gpu(c.table), gpu(np.array([0, n], np.int32)), gpu(c.lengths)
    q = fused[:, :heads * per]
    out = torch.empty((n, heads * per, dim), device="cuda", dtype=torch.float16)
    assert qmm.cache_attention(*args, q, *batch, out=out) is out
    assert torch.equal(out, qmm.cache_attention(*args, q.contiguous(), *batch))


def test_parts_of_a_sequence_join_by_lse():
    """Two halves of a context, attended to apart and joined, give the whole: what lse is for."""
    heads, per, dim, n = 2, 2, 64, 256
    c = ref.Cache(90, 8, 8, heads, dim, 64, [n])
    q = torch.randn((1, heads * per, dim), device="cuda")
    kc, vc, one = gpu(c.k_cache), gpu(c.v_cache), gpu(np.array([0, 1], np.int32))
    parts = []
    for table, length in ((c.table[:, :2], 128), (c.table[:, 2:], 128), (c.table, 256)):
        lse = torch.empty((1, heads * per), device="cuda")
        o = qmm.cache_attention(8, 8, kc, vc, q, gpu(table), one, gpu(np.array([length], np.int32)), causal=False, lse=lse)
        parts.append((o.double(), lse.double()))
    (a, la), (b, lb), (w, lw) = parts
    total = torch.logaddexp(la, lb)
    joined = a * torch.exp(la - total)[..., None] + b * torch.exp(lb - total)[..., None]
    # both sides are the same formula with f32 errors of at most 2^-17 at these sizes (see above), values below 5
    assert (joined - w).abs().max() < 5 * 2.0**-16 and (total - lw).abs().max() < 2.0**-16
