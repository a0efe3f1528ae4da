"""Attention of many rows with work for the whole card (over 512 row tiles of
16, from 192 rows of a sequence: keys and values are decoded once for 128 or 256
rows), and batches of up to 64 sequences with rows in any of them.  Tolerances
as for few rows: there f16 rows allow for a probability of one part, here they
have two, and values are rounded.
"""
import numpy as np
import pytest

import cache_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_matmul_gguf_amd as qmm  # noqa: E402
from test_gpu_attention import FMTS, TYPES, check, gpu, largest, run_case, slack, starts_of  # noqa: E402

FORMATS = [("q8", "q8"), ("q4", "q4"), ("q8", "q4"), ("q4", "q8")]
WIDE = ([300, 70, 0, 129], [70, 70, 0, 60])     # 400 rows on average: as many in tiles of 256 as of 128
NARROW = ([200, 75, 77], [76, 75, 77])          # 608: fewer empty rows in tiles of 128


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fk,fv", FORMATS)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("lengths,new", [WIDE, NARROW])
def test_every_format(lengths, new, dim, fk, fv, dtype):
    print(f"every format {lengths} {new} {dim} {fk} {fv} {dtype}", flush=True)
    run_case(200 + dim, fk, fv, dtype, 8, 8, dim, 64, lengths, new)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fk,fv,dim", [("q8", "q8", 128), ("q4", "q8", 64), ("q8", "q4", 256)])
@pytest.mark.parametrize("kw", [dict(window=1), dict(window=65), dict(softcap=20.0, q_scale=8.0), dict(softcap=5.0, window=33),
                                dict(causal=False), dict(scale=0.0), dict(scale=-0.1)], ids=str)
@pytest.mark.parametrize("lengths,new", [WIDE, NARROW])
def test_masks_and_scores(lengths, new, kw, fk, fv, dim, dtype):
    print(f"masks {lengths} {new} {kw} {fk} {fv} {dim} {dtype}", flush=True)
    run_case(230, fk, fv, dtype, 8, 8, dim, 128, lengths, new, **kw)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(window=700), dict(max_length=1500), dict(max_length=600)], ids=str)
def test_pieces(kw, dim, dtype):
    a = run_case(240, "q8", "q4", dtype, 32, 8, dim, 64, [1500, 800], [25, 25], **kw)
    b = run_case(240, "q8", "q4", dtype, 32, 8, dim, 64, [1500, 800], [25, 25], **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fk,fv", [("q8", "q8"), ("q4", "q4")])
@pytest.mark.parametrize("dim", [64, 128])
def test_values_that_are_not_finite(dim, fk, fv, dtype):
    n, heads, per, new = 200, 14, 8, 80
    c = ref.Cache(260, FMTS[fk], FMTS[fv], heads, dim, 64, [n])
    c.v[0][n - 2, 0, 40] = np.nan
    c.v[0][10, 1, 3] = np.inf
    c.write()
    run_case(260, fk, fv, dtype, heads, per, dim, 64, [n], [new], cache=c, window=150)
    c.k[0][n - 1, 2, 5] = np.inf
    c.write()
    run_case(260, fk, fv, dtype, heads, per, dim, 64, [n], [new], cache=c, window=150)
    q = torch.randn((new, heads * per, dim), device="cuda").to(TYPES[dtype])
    q[0, 0, 7] = float("nan")
    q[1, 9, 9] = float("inf")
    c = ref.Cache(261, FMTS[fk], FMTS[fv], heads, dim, 64, [n])
    out = qmm.cache_attention(c.fmt_k, c.fmt_v, gpu(c.k_cache), gpu(c.v_cache), q, gpu(c.table),
                              gpu(np.array([0, new], np.int32)), gpu(c.lengths))
    bad = torch.isnan(out)
    assert bad[0, 0].all() and bad[1, 9].all() and int(bad.any(2).sum()) == 2


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fk,fv", [("q8", "q8"), ("q4", "q4")])
def test_the_ends_of_the_range(fk, fv, dtype):
    n, dim, heads, per, new = 300, 64, 14, 8, 80
    for v_scale, q_scale, mixed in ((1e-3, 1.0, False), (6e3, 1.0, False), (1.0, 1e-3, False), (1.0, 30.0, False), (1.0, 1.0, True)):
        c = ref.Cache(270, FMTS[fk], FMTS[fv], heads, dim, 64, [n], v_scale=v_scale)
        if mixed:
            c.v[0] *= np.exp2(np.random.default_rng(5).integers(-8, 9, (n, 1, 1))).astype(np.float32)
            c.k[0] *= np.exp2(np.random.default_rng(6).integers(-6, 3, (n, 1, 1))).astype(np.float32)
            c.write()
        run_case(271, fk, fv, dtype, heads, per, dim, 64, [n], [new], cache=c, q_scale=q_scale)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rows_and_pages_that_are_not_there(dtype):
    """Rows of no sequence stay, rows before position 0 are zeros, pages without an entry are not seen."""
    dt, heads, per, dim, page = TYPES[dtype], 8, 8, 128, 64
    c = ref.Cache(280, 8, 2, heads, dim, page, [20, 400, 64 * 15])
    new = [60, 70, 80]
    gone = [0, 1, 5, 14]
    c.table[2, gone] = [-1, 10**6, -2**31, 2**31 - 1]
    st = 3 + starts_of(new)
    t = int(st[-1]) + 5
    q = torch.from_numpy(np.random.default_rng(3).standard_normal((t, heads * per, dim)).astype(np.float32)).to(dt)
    for window in (0, 100):
        out = torch.full((t, heads * per, dim), 7.0, device="cuda", dtype=dt)
        lse = torch.full((t, heads * per), 7.0, device="cuda")
        qmm.cache_attention(8, 2, gpu(c.k_cache), gpu(c.v_cache), q.cuda(), gpu(c.table), gpu(st), gpu(c.lengths), window=window,
                            out=out, lse=lse)
        for rows in (slice(0, 3), slice(int(st[-1]), t)):
            assert (out[rows] == 7).all() and (lse[rows] == 7).all()
        for s, n in enumerate(c.lengths):
            rows = slice(st[s], st[s + 1])
            seen = ~np.isin(np.arange(n) // page, gone) if s == 2 else None
            o, l, big, top = ref.attention(q[rows].double().numpy(), c.kq[s], c.vq[s], np.arange(n - new[s], n), dim ** -0.5,
                                           window=window, seen=seen)
            check(out[rows], o, slack(dt, dim, n, big, top, largest(c.vq[s]))[0], f"window {window}, sequence {s}")
            assert np.array_equal(np.isneginf(lse[rows].cpu().numpy()), np.isneginf(l))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("count", [2, 16, 17, 31, 33, 47, 49, 63, 64])
@pytest.mark.parametrize("most", [1, 3, 40])
def test_sequences_of_any_number_of_rows(most, count, dtype):
    """Which sequence a tile is of: batches up to a wave's lanes, with and without rows."""
    rng = np.random.default_rng(count)
    new = [int(x) for x in rng.integers(0, most + 1, count)]
    new[-1] = 1
    lengths = [int(x) for x in np.maximum(new, rng.integers(1, 150, count))]
    run_case(290, "q8", "q8", dtype, 2, 3, 64, 64, lengths, new)
