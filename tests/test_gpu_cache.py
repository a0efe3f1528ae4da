"""The quantized paged cache on the GPU: bytes that are stored and values that
are read back, against GGUF blocks of the oracle's quantizers.  Both are exact:
codes and scales follow f32 steps that the format's rule fixes, and a value is
one product of an f16 scale and a code of at most 8 bits, exact in f32 and
rounded once to the output's type."""
import numpy as np
import pytest

import cache_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_matmul_gguf_amd as qmm  # noqa: E402

FMTS = {"q8": qmm.Q8_0, "q4": qmm.Q4_0}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    qmm.lib()


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def starts_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def same(a, b, what):
    """Equal values, NaN equal to NaN, zeros of either sign."""
    a, b = a.detach().cpu().double().numpy(), b.detach().cpu().double().numpy()
    bad = ~((a == b) | (np.isnan(a) & np.isnan(b)))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} differ, first at {tuple(np.argwhere(bad)[0])}"


def typed(x, dt):
    """f32 numpy -> (the GPU tensor of type dt, the f32 values it holds)."""
    t = torch.from_numpy(x).to(dt)
    return t.cuda(), t.float().numpy()


# lengths, new tokens, page size
BATCHES = [
    ([1], [1], 64), ([307], [1], 64), ([64, 65, 128, 1], [1, 1, 1, 1], 64), ([70, 3, 200], [70, 3, 200], 128),
    ([130, 40, 64, 500], [7, 0, 64, 261], 64), ([1000], [999], 256), ([90, 300, 17], [33, 17, 16], 192),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fk,fv", [("q8", "q8"), ("q4", "q4"), ("q8", "q4"), ("q4", "q8")])
@pytest.mark.parametrize("heads,dim", [(3, 64), (2, 96), (1, 128), (2, 256)])
@pytest.mark.parametrize("lengths,new,page", BATCHES)
def test_store_and_load(lengths, new, page, heads, dim, fk, fv, dtype):
    print(f"store {lengths} {new} {page} {heads}x{dim} {fk} {fv} {dtype}", flush=True)
    dt = TYPES[dtype]
    old = [n - m for n, m in zip(lengths, new)]
    c = ref.Cache(7, FMTS[fk], FMTS[fv], heads, dim, page, lengths)
    want_k, want_v = c.k_cache, c.v_cache
    pool = ref.Cache(7, FMTS[fk], FMTS[fv], heads, dim, page, lengths)  # the same garbage and old tokens
    rng = np.random.default_rng(8)
    t = sum(new)
    st = starts_of(new)
    k, kv = typed(rng.standard_normal((t, heads, dim)).astype(np.float32), dt)
    v, vv = typed((3 * rng.standard_normal((t, heads, dim))).astype(np.float32), dt)
    for s, n in enumerate(lengths):
        c.k[s][old[s]:] = kv[st[s]:st[s + 1]]
        c.v[s][old[s]:] = vv[st[s]:st[s + 1]]
    c.write()
    kc, vc = gpu(pool.k_cache), gpu(pool.v_cache)
    args = FMTS[fk], FMTS[fv], kc, vc
    batch = gpu(c.table), gpu(st), gpu(c.lengths)
    qmm.cache_store(*args, k, v, *batch)
    assert np.array_equal(kc.cpu().numpy(), want_k), "keys' bytes"
    assert np.array_equal(vc.cpu().numpy(), want_v), "values' bytes"
    # the new tokens and whole sequences read back
    whole = gpu(starts_of(lengths))
    for out_dt in TYPES.values():
        for b, rows in (((batch[0], batch[1], batch[2]), old), ((batch[0], whole, batch[2]), [0] * len(lengths))):
            gk, gv = qmm.cache_load(*args, *b, tokens=int(b[1][-1]), dtype=out_dt)
            for got, vals, what in ((gk, c.kq, "keys"), (gv, c.vq, "values")):
                same(got, torch.from_numpy(np.concatenate([x[o:] for x, o in zip(vals, rows)])).to(out_dt), what)


def test_rows_and_positions_without_a_place():
    """Rows before the first and behind the last sequence, positions before a sequence and past its table, and entries
    that name no page: nothing is written for them, zeros come back, other bytes stay."""
    heads, dim, page = 2, 64, 64
    rng = np.random.default_rng(3)
    kc = rng.integers(0, 256, (5, heads, page, ref.row_bytes(8, dim)), dtype=np.uint8)
    vc = rng.integers(0, 256, (5, heads, page, ref.row_bytes(2, dim)), dtype=np.uint8)
    table = np.array([[3, 5], [-1, 1], [0, 2**31 - 1], [2, 4]], dtype=np.int32)  # 5, -1 and 2^31 - 1 name no page
    lengths = np.array([80, 70, 65, 140], dtype=np.int32)  # the last passes its table
    starts = np.array([3, 103, 123, 130, 150], dtype=np.int32)  # 100 (20 before position 0), 20, 7 and 20 rows
    t = 160
    k, kv = typed(rng.standard_normal((t, heads, dim)).astype(np.float32), torch.float32)
    v, vv = typed(rng.standard_normal((t, heads, dim)).astype(np.float32), torch.float32)
    want_k, want_v = kc.copy(), vc.copy()
    back_k, back_v = np.full((t, heads, dim), 7.0), np.full((t, heads, dim), 7.0)
    for s in range(4):
        for n in range(starts[s], starts[s + 1]):
            pos = lengths[s] - (starts[s + 1] - n)
            p = table[s, pos // page] if 0 <= pos < 2 * page else -1
            for h in range(heads):
                for fmt, vals, cache, x, back in ((8, False, want_k, kv, back_k), (2, True, want_v, vv, back_v)):
                    q, d = ref.quantize(fmt, x[n, h])
                    back[n, h] = 0
                    if 0 <= p < 5:
                        ref.write(cache, fmt, vals, p, h, pos % page, q, d)
                        back[n, h] = ref.values(q, d)
    kd, vd = gpu(kc), gpu(vc)
    args = qmm.Q8_0, qmm.Q4_0, kd, vd
    batch = gpu(table), gpu(starts), gpu(lengths)
    qmm.cache_store(*args, k, v, *batch)
    assert np.array_equal(kd.cpu().numpy(), want_k) and np.array_equal(vd.cpu().numpy(), want_v)
    gk = torch.full((t, heads, dim), 7.0, device="cuda")
    gv = torch.full((t, heads, dim), 7.0, device="cuda")
    qmm.cache_load(*args, *batch, tokens=t, k=gk, v=gv)
    same(gk, torch.from_numpy(back_k), "keys")
    same(gv, torch.from_numpy(back_v), "values")


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_the_ends_of_the_range(fmt, dtype):
    """Blocks of zeros, of tiny and of large values, ties, one infinity or NaN among fine values."""
    f, dt, dim, page = FMTS[fmt], TYPES[dtype], 64, 64
    top = float(torch.finfo(dt).max)
    rng = np.random.default_rng(5)
    rows = [np.zeros(dim), np.full(dim, 1e-3), rng.standard_normal(dim) * 1e-6, rng.standard_normal(dim) * 1e-9,
            np.full(dim, min(top, 65504.0)), rng.standard_normal(dim) * 2e4]
    for sign in (1, -1):
        x = np.repeat([1.0, -1.0], 32) * sign  # both signs reach the largest magnitude
        x[::3] *= -1
        rows.append(x)
    x = np.arange(64) % 32 - 16.0
    rows += [x, -x, x / 127, x * 0.5 / 127]
    for bad in (np.inf, -np.inf, np.nan):
        x = rng.standard_normal(dim)
        x[37] = bad
        rows.append(x)
    if dtype != "f16":
        for big in (8e6, 9e6, 3e38, 5.2e5, 5.3e5, 1e-30, 1e-44):
            x = rng.standard_normal(dim)
            x[5], x[40] = big, -big
            x[41:] = 0
            rows.append(x)
    x32 = np.array(rows, dtype=np.float64)[:, None, :]
    k, kv = typed(x32.astype(np.float32), dt)
    n = len(rows)
    q, d = ref.quantize(f, kv)
    want = ref.values(q, d)
    shape = (1, 1, page, ref.row_bytes(f, dim))
    kc, vc = torch.zeros(shape, dtype=torch.uint8, device="cuda"), torch.zeros(shape, dtype=torch.uint8, device="cuda")
    batch = gpu(np.zeros((1, 1), np.int32)), gpu(np.array([0, n], np.int32)), gpu(np.array([n], np.int32))
    qmm.cache_store(f, f, kc, vc, k, k, *batch)
    ek, ev = np.zeros(shape, np.uint8), np.zeros(shape, np.uint8)
    for t in range(n):
        ref.write(ek, f, False, 0, 0, t, q[t, 0], d[t, 0])
        ref.write(ev, f, True, 0, 0, t, q[t, 0], d[t, 0])
    gk, gv = qmm.cache_load(f, f, kc, vc, *batch, tokens=n)
    same(gk, torch.from_numpy(want), "keys")
    same(gv, torch.from_numpy(want), "values")
    fine = np.isfinite(want).all()
    if fine:
        assert np.array_equal(kc.cpu().numpy(), ek) and np.array_equal(vc.cpu().numpy(), ev)


@pytest.mark.parametrize("fk,fv", [("q8", "q4"), ("q4", "q8")])
def test_strided_tokens(fk, fv):
    """k and v as parts of one tensor of a fused product's outputs."""
    heads, dim, page, n = 2, 96, 64, 150
    c = ref.Cache(11, FMTS[fk], FMTS[fv], heads, dim, page, [n])
    rng = np.random.default_rng(12)
    fused = torch.from_numpy(rng.standard_normal((n, 5 * heads, dim)).astype(np.float32)).to(torch.bfloat16).cuda()
    k, v = fused[:, 3 * heads:4 * heads], fused[:, 4 * heads:]
    pool = gpu(c.k_cache), gpu(c.v_cache)
    other = pool[0].clone(), pool[1].clone()
    batch = gpu(c.table), gpu(np.array([0, n], np.int32)), gpu(c.lengths)
    qmm.cache_store(FMTS[fk], FMTS[fv], *pool, k, v, *batch)
    qmm.cache_store(FMTS[fk], FMTS[fv], *other, k.contiguous(), v.contiguous(), *batch)
    assert torch.equal(pool[0], other[0]) and torch.equal(pool[1], other[1])


def test_blocks_are_those_of_the_activation_quantizer():
    heads, dim, n = 4, 128, 64
    x = torch.randn((n, heads, dim), device="cuda")
    blocks = qmm.quantize_act(qmm.Q8_0, x.view(n * heads, dim))
    want = qmm.dequantize_weights(qmm.Q8_0, blocks, n * heads, dim).view(n, heads, dim)
    shape = (1, heads, 64, qmm.row_bytes(qmm.Q8_0, dim))
    kc, vc = torch.zeros(shape, dtype=torch.uint8, device="cuda"), torch.zeros(shape, dtype=torch.uint8, device="cuda")
    batch = gpu(np.zeros((1, 1), np.int32)), gpu(np.array([0, n], np.int32)), gpu(np.array([n], np.int32))
    qmm.cache_store(qmm.Q8_0, qmm.Q8_0, kc, vc, x, x, *batch)
    k, v = qmm.cache_load(qmm.Q8_0, qmm.Q8_0, kc, vc, *batch, tokens=n)
    assert torch.equal(k, want) and torch.equal(v, want)


def test_a_pool_past_32_bits():
    """Pages whose bytes lie past 2^32 in both pools."""
    heads, dim, page = 8, 128, 256
    pages = (9 << 29) // (heads * page * ref.row_bytes(8, dim))
    shape = (pages, heads, page, ref.row_bytes(8, dim))
    kc = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    assert kc.numel() > 1 << 32
    n = 300
    k, kv = typed(np.random.default_rng(1).standard_normal((n, heads, dim)).astype(np.float32), torch.float32)
    batch = gpu(np.array([[pages - 1, 0]], np.int32)), gpu(np.array([0, n], np.int32)), gpu(np.array([n], np.int32))
    qmm.cache_store(qmm.Q8_0, qmm.Q8_0, kc, vc, k, -k, *batch)
    gk, gv = qmm.cache_load(qmm.Q8_0, qmm.Q8_0, kc, vc, *batch, tokens=n)
    want = torch.from_numpy(ref.values(*ref.quantize(8, kv)))
    same(gk, want, "keys")
    same(gv, -want, "values")
    assert int(kc[1:-1].count_nonzero()) == 0 and int(vc[1:-1].count_nonzero()) == 0
    q = torch.randn((1, heads, dim), device="cuda")
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out = qmm.cache_attention(qmm.Q8_0, qmm.Q8_0, kc, vc, q, batch[0], one, batch[2])
    o, _, big, top = ref.attention(q.cpu().double().numpy(), want.numpy(), -want.numpy(), [n - 1], dim ** -0.5)
    err = np.abs(out.cpu().double().numpy() - o)
    assert (err <= big * (2.0**-18 * (1 + top.max()))).all()
