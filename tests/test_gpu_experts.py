"""Mixture-of-experts calls and 4-bit group products on the GPU against plain
implementations in 64 bits.

Tolerance of a product with the exact value y and A = sum_k |w_k x_k| (for
Q4_K, whose values are differences, with |d sc q| + |dmin m| for |w|):
  * sums are carried in f32 in blocks: a block of at most 256 products, then
    one addition per block (at most K / 32 blocks).  At the sizes below (K <=
    4096) that is under 168 additions in a chain, each off by at most 2^-24 of
    a partial sum no larger than A: under 1e-5 A, the library's bar;
  * one rounding to the output type: half a step, eps/2 of the rounded value
    (plus half the type's smallest step for values below its normal range).
h = act(g) u: |act'| <= 1.13, |act(v)| <= |v|, and the f32 activation itself is
good to 2^-20 of its value (exp's argument and result rounding, |g| < 16).
"""
import math

import numpy as np
import pytest

import oracle
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_matmul_gguf_amd as qmm  # noqa: E402

BAR = 1e-5
FMTS = {"Q8_0": qmm.Q8_0, "Q4_0": qmm.Q4_0, "Q5_0": qmm.Q5_0, "Q4_K": qmm.Q4_K, "Q6_K": qmm.Q6_K}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {torch.float32: 2.0**-150, torch.float16: 2.0**-25, torch.bfloat16: 2.0**-134}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    qmm.lib()


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, want, slack, what):
    """|got - want| within slack (absolute, per element) and one rounding to got's type."""
    eps = torch.finfo(got.dtype).eps / 2
    g = f64(got)
    tol = slack + eps * (np.abs(want) + slack) + TINY[got.dtype]
    bad = ~(np.abs(g - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {g[i]!r} want {want[i]!r} tol {tol[i]!r}")


def weights_of(fmt, seed, rows, k):
    """(blocks uint8 [rows, bytes], W f64, |W| as summed f64)"""
    b = oracle.quantize(fmt, synth.weights_f32(seed, rows, k))
    w = oracle.dequantize(fmt, b, k)
    return b, w, magnitude(fmt, b, w, k)


def magnitude(fmt, b, w, k):
    if fmt != qmm.Q4_K:
        return np.abs(w)
    low = b.copy().reshape(len(b), -1, 144)
    low[:, :, 2:4] = 0  # dmin = 0: the values before the minimum is taken off
    low = oracle.dequantize(fmt, low.reshape(len(b), -1), k)
    return np.abs(low) + np.abs(low - w)


def acts(seed, shape, dtype, scale=1.0):
    x = torch.from_numpy(synth.acts_f32(seed, int(np.prod(shape[:-1])), shape[-1], scale).reshape(shape)).to(dtype)
    return x.cuda(), x.double().numpy()


def choose(seed, t, e, k, how):
    g = np.random.default_rng(seed)
    if how == "same":  # every pair on one expert
        ids = np.full((t, k), int(g.integers(e)))
    elif how == "twice":  # repeats within a token, and no-expert slots of several kinds
        ids = g.integers(0, e, (t, k))
        ids[g.random((t, k)) < 0.2] = -1
        ids[g.random((t, k)) < 0.1] = e
        ids[0, 0] = 2**31 - 1
        ids[-1, :] = -2**31
    else:
        ids = np.stack([g.permutation(e)[:k] if k <= e else g.integers(0, e, k) for _ in range(t)])
    return ids.astype(np.int32)


def product_ref(w, wa, e, n, ids, x):
    """x [T, k, K] f64 -> (y, A) [T, k, n]; zeros without an expert."""
    t, k = ids.shape
    y, a = np.zeros((t, k, n)), np.zeros((t, k, n))
    for i in range(e):
        at = ids == i
        if at.any():
            y[at] = x[at] @ w[i * n:(i + 1) * n].T
            a[at] = np.abs(x[at]) @ wa[i * n:(i + 1) * n].T
    return y, a


def per_slot(x, k):
    return np.repeat(x[:, None, :], k, 1)


# (T, E, k, N, K multiple, choice): one token, few, a tile's edge, long ones
SHAPES = [
    (1, 4, 2, 16, 1, "any"), (1, 64, 8, 97, 2, "any"), (1, 3, 3, 33, 6, "same"), (2, 5, 1, 130, 3, "twice"),
    (5, 8, 3, 64, 2, "any"), (17, 4, 2, 40, 1, "twice"), (16, 2, 1, 96, 5, "same"), (33, 16, 4, 48, 2, "any"),
    (130, 3, 2, 65, 2, "twice"), (300, 8, 2, 128, 3, "any"), (257, 5, 3, 31, 1, "same"), (129, 40, 4, 16, 2, "any"),
]


def k_of(fmt, mult):
    return mult * (256 if fmt in (qmm.Q4_K, qmm.Q6_K) else (32, 64, 96, 160, 192, 288)[mult - 1])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("t,e,k,n,mult,how", SHAPES)
def test_experts_products(fmt, dtype, t, e, k, n, mult, how):
    print(f"experts {fmt} {dtype} T={t} E={e} k={k} N={n} mult={mult} {how}", flush=True)
    f, dt = FMTS[fmt], TYPES[dtype]
    kk = k_of(f, mult)
    b, w, wa = weights_of(f, 10 + t + n, e * n, kk)
    wd = torch.from_numpy(b.reshape(e, n, -1)).cuda()
    ids_h = choose(20 + t, t, e, k, how)
    ids = torch.from_numpy(ids_h).cuda()
    x, xh = acts(30 + t, (t, kk), dt)
    y, a = product_ref(w, wa, e, n, ids_h, per_slot(xh, k))
    close(qmm.experts_matmul(f, wd, x, ids), y, BAR * a, "experts_matmul")

    h, hh = acts(31 + t, (t, k, kk), dt)
    y, a = product_ref(w, wa, e, n, ids_h, hh)
    close(qmm.experts_matmul(f, wd, h, ids), y, BAR * a, "experts_matmul per slot")

    g = np.random.default_rng(40 + t).random((t, k)).astype(np.float32)
    got = qmm.experts_combine(f, wd, h, ids, torch.from_numpy(g).cuda())
    gd = g.astype(np.float64)[:, :, None]
    close(got, (y * gd).sum(1), BAR * (a * gd).sum(1), "experts_combine")


def act_ref(v, act):
    if act == "silu":
        return v / (1 + np.exp(-v))
    return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v**3)))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("t,e,k,n,mult,how", SHAPES)
def test_experts_glu(fmt, dtype, act, t, e, k, n, mult, how):
    print(f"glu {fmt} {dtype} {act} T={t} E={e} k={k} N={n} mult={mult} {how}", flush=True)
    f, dt = FMTS[fmt], TYPES[dtype]
    kk = k_of(f, mult)
    b0, w0, a0 = weights_of(f, 11 + t + n, e * n, kk)
    b1, w1, a1 = weights_of(f, 12 + t + n, e * n, kk)
    ids_h = choose(21 + t, t, e, k, how)
    x, xh = acts(32 + t, (t, kk), dt)
    got = qmm.experts_glu(f, torch.from_numpy(b0.reshape(e, n, -1)).cuda(), torch.from_numpy(b1.reshape(e, n, -1)).cuda(),
                          x, torch.from_numpy(ids_h).cuda(), act=act)
    xs = per_slot(xh, k)
    g, ga = product_ref(w0, a0, e, n, ids_h, xs)
    u, ua = product_ref(w1, a1, e, n, ids_h, xs)
    ag = act_ref(g, act)
    eg, eu = BAR * ga, BAR * ua
    slack = 1.13 * eg * (np.abs(u) + eu) + np.abs(g) * eu + 2.0**-20 * np.abs(ag * u)
    close(got, ag * u, slack, "experts_glu")


# ----------------------------------------------------------------- w4 -----

def w4_case(seed, n, k, group, zeros, sdtype):
    g = np.random.default_rng(seed)
    codes = g.integers(0, 16, (n, k))
    q = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    s = torch.from_numpy((0.01 * (g.random((n, k // group)) - 0.3)).astype(np.float32)).to(sdtype)
    z = g.integers(0, 16, (n, k // group)).astype(np.uint8) if zeros else None
    zz = np.repeat(z.astype(np.int64), group, 1) if zeros else 8
    w = (codes - zz) * np.repeat(s.double().numpy(), group, 1)
    return torch.from_numpy(q).cuda(), s.cuda(), None if z is None else torch.from_numpy(z).cuda(), w


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,n,k,group,zeros,sdtype", [
    (1, 1, 32, 32, False, "f16"), (1, 16, 128, 128, True, "f32"), (1, 577, 1536, 64, False, "bf16"),
    (2, 33, 96, 32, True, "f16"), (3, 1000, 576, 576, False, "f16"), (5, 64, 4096, 128, True, "f16"),
    (8, 200, 160, 32, False, "f32"), (9, 96, 1024, 256, True, "bf16"), (16, 49, 288, 96, True, "f16"),
    (17, 130, 640, 64, False, "f16"), (33, 64, 512, 512, True, "f32"), (70, 257, 224, 32, True, "f16"),
    (128, 128, 384, 128, False, "bf16"), (300, 100, 1536, 32, True, "f16"), (513, 385, 256, 64, True, "f16"),
])
def test_w4(dtype, m, n, k, group, zeros, sdtype):
    print(f"w4 {dtype} M={m} N={n} K={k} G={group} zeros={zeros} {sdtype}", flush=True)
    q, s, z, w = w4_case(50 + m, n, k, group, zeros, TYPES[sdtype])
    x, xh = acts(60 + m, (m, k), TYPES[dtype])
    close(qmm.w4_matmul(q, s, x, zeros=z), xh @ w.T, BAR * (np.abs(xh) @ np.abs(w).T), "w4")


def test_w4_zero_points_beyond_a_nibble():
    q, s, z, w = w4_case(70, 40, 256, 64, True, torch.float16)
    far = torch.from_numpy(np.random.default_rng(71).integers(0, 256, (40, 4)).astype(np.uint8)).cuda()
    codes = np.stack([(q.cpu().numpy() & 15), q.cpu().numpy() >> 4], -1).reshape(40, 256).astype(np.float64)
    w = (codes - np.repeat(f64(far), 64, 1)) * np.repeat(f64(s), 64, 1)
    for m in (1, 20, 200):
        x, xh = acts(72, (m, 256), torch.float32)
        close(qmm.w4_matmul(q, s, x, zeros=far), xh @ w.T, BAR * (np.abs(xh) @ np.abs(w).T), "w4")


# ------------------------------------------------------- hard activations --

def value_rows(k):
    """Rows of activations whose sizes differ widely, within a row and between rows (f32)."""
    g = np.random.default_rng(80)
    x = g.standard_normal((24, k)).astype(np.float32)
    x[1] = 0
    x[2] *= 1e30
    x[3] *= 1e-30
    x[4] *= np.float32(10.0) ** g.integers(-12, 12, k)
    x[5, :] = 0
    x[5, k // 2] = 3.0
    x[6, ::7] *= 1e20
    x[7, :k // 2] *= 1e-25
    x[8] *= 2.0**-140  # below f32's normal range
    x[9] *= 60000
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", list(FMTS) + ["W4"])
@pytest.mark.parametrize("rows", [1, 12, 24 * 12])
def test_wide_ranges(fmt, dtype, rows):
    k, n = 512, 37
    base = value_rows(k)
    x = torch.from_numpy(np.tile(base, (max(1, rows // 24), 1))).to(TYPES[dtype])
    picks = range(24) if rows == 1 else [slice(0, rows)]
    if fmt == "W4":
        q, s, z, w = w4_case(81, n, k, 64, True, torch.float16)
        wa = np.abs(w)
        call = lambda v: qmm.w4_matmul(q, s, v, zeros=z)  # noqa: E731
    else:
        b, w, wa = weights_of(FMTS[fmt], 82, n, k)
        wd = torch.from_numpy(b.reshape(1, n, -1)).cuda()
        call = lambda v: qmm.experts_matmul(FMTS[fmt], wd, v, torch.zeros((len(v), 1), dtype=torch.int32).cuda())[:, 0]  # noqa: E731
    for p in picks:
        xs = x[p].reshape(-1, k)
        xh = xs.double().numpy()
        # values below 2^-126 may be taken as zero (a product's f32 sum cannot hold them)
        floor = 2.0**-126 * k * wa.max()
        with np.errstate(over="ignore"):
            close(call(xs.cuda()), xh @ w.T, BAR * (np.abs(xh) @ wa.T) + floor, f"rows {p}")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMTS) + ["W4"])
@pytest.mark.parametrize("m", [1, 12, 300])
def test_non_finite_rows_stay_in_their_rows(fmt, dtype, m):
    k, n = 512, 33
    x, _ = acts(90, (m, k), TYPES[dtype])
    bad = {0: float("nan")} if m == 1 else {0: float("nan"), 3: float("inf"), m - 1: float("-inf")}
    for r, v in bad.items():
        x[r, (37 * r) % k] = v
    if fmt == "W4":
        q, s, z, w = w4_case(91, n, k, 64, False, torch.float16)
        y = qmm.w4_matmul(q, s, x)
        wa = np.abs(w)
    else:
        b, w, wa = weights_of(FMTS[fmt], 92, n, k)
        y = qmm.experts_matmul(FMTS[fmt], torch.from_numpy(b.reshape(1, n, -1)).cuda(), x,
                               torch.zeros((m, 1), dtype=torch.int32).cuda())[:, 0]
    fin = torch.isfinite(y).cpu().numpy()
    good = [r for r in range(m) if r not in bad]
    for r in bad:
        assert not fin[r].any()
    if good:
        xh = f64(x)[good]
        close(y[good], xh @ w.T, BAR * (np.abs(xh) @ wa.T), "finite rows")


def test_no_expert_slots_ignore_what_they_hold():
    f, e, n, k, t = qmm.Q8_0, 4, 40, 64, 6
    b, w, wa = weights_of(f, 95, e * n, k)
    wd = torch.from_numpy(b.reshape(e, n, -1)).cuda()
    for reps in (1, 60):
        ids_h = np.tile(choose(96, t, e, 3, "any"), (reps, 1))
        ids_h[2] = -1
        ids_h[4, 1] = e + 5
        h, hh = acts(97, (t * reps, 3, k), torch.float32)
        g = torch.rand((t * reps, 3)).cuda()
        h[2], g[2] = float("nan"), float("inf")
        h[4, 1], g[4, 1] = float("inf"), float("nan")
        hh = hh.copy()
        hh[2], hh[4, 1] = 0, 0
        gh = f64(g)
        gh[2], gh[4, 1] = 0, 0
        y, a = product_ref(w, wa, e, n, ids_h, hh)
        got = qmm.experts_combine(f, wd, h, torch.from_numpy(ids_h).cuda(), g)
        close(got, (y * gh[..., None]).sum(1), BAR * (a * gh[..., None]).sum(1), "combine")
        assert (got[2] == 0).all()
        slots = qmm.experts_matmul(f, wd, h, torch.from_numpy(ids_h).cuda())
        assert (slots[2] == 0).all() and (slots[4, 1] == 0).all()


def test_empty_batches():
    b, _, _ = weights_of(qmm.Q4_0, 98, 8, 64)
    wd = torch.from_numpy(b.reshape(2, 4, -1)).cuda()
    ids = torch.zeros((0, 2), dtype=torch.int32).cuda()
    assert qmm.experts_matmul(qmm.Q4_0, wd, torch.zeros((0, 64)).cuda(), ids).shape == (0, 2, 4)
    assert qmm.experts_glu(qmm.Q4_0, wd, wd, torch.zeros((0, 64)).cuda(), ids).shape == (0, 2, 4)
    assert qmm.experts_combine(qmm.Q4_0, wd, torch.zeros((0, 2, 64)).cuda(), ids, torch.zeros((0, 2)).cuda()).shape == (0, 4)
    assert qmm.route_experts(torch.zeros((0, 8)).cuda(), 2)[0].shape == (0, 2)
    q, s, z, _ = w4_case(99, 5, 64, 32, False, torch.float16)
    assert qmm.w4_matmul(q, s, torch.zeros((0, 64)).cuda()).shape == (0, 5)


# --------------------------------------------------------------- router ---

def route_ref(l, k, score, bias, groups, top_groups, group_top, renorm, scale):
    t, e = l.shape
    ids, ws = np.full((t, k), -1, np.int32), np.zeros((t, k))
    for r in range(t):
        row = [float(v) for v in l[r]]
        live = [i for i in range(e) if not math.isnan(row[i]) and row[i] != -math.inf]
        if score == "softmax":
            top = max((row[i] for i in live), default=0.0)
            p = {i: 1.0 if row[i] == top else math.exp(row[i] - top) for i in live}
            tot = math.fsum(p.values())
            s = {i: p[i] / tot for i in live}
        else:
            s = {i: 1 / (1 + math.exp(-row[i])) if row[i] > -700 else 0.0 for i in live}
        c = {i: s[i] + (float(bias[i]) if bias is not None else 0.0) for i in live}
        c = {i: v for i, v in c.items() if not math.isnan(v) and v != -math.inf}
        if groups > 1:
            size, sc = e // groups, {}
            for i, v in c.items():
                sc.setdefault(i // size, []).append(v)
            order = sorted(sc, key=lambda g: (-sum(sorted(sc[g])[::-1][:group_top]), g))[:top_groups]
            c = {i: v for i, v in c.items() if i // size in order}
        pick = sorted(c, key=lambda i: (-c[i], i))[:k]
        w = [s[i] for i in pick]
        if renorm:
            tot = math.fsum(w)
            w = [v / tot if tot > 0 else 0.0 for v in w]
        ids[r, :len(pick)] = pick
        ws[r, :len(pick)] = [v * scale for v in w]
    return ids, ws


ROUTES = [
    (1, 64, 8, "softmax", False, 1, 1, 1, True, 1.0), (1, 1, 1, "sigmoid", True, 1, 1, 1, True, 2.0),
    (5, 2, 2, "softmax", True, 2, 1, 1, False, 1.0), (7, 65, 5, "sigmoid", True, 5, 2, 2, True, 2.5),
    (33, 128, 64, "softmax", False, 1, 1, 1, False, 1.0), (19, 160, 6, "softmax", False, 8, 3, 1, False, 16.0),
    (40, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5), (3, 512, 10, "softmax", True, 64, 3, 2, True, 1.0),
    (9, 1000, 16, "sigmoid", False, 50, 7, 1, True, 1.0), (4, 1024, 64, "softmax", True, 1, 1, 1, True, 1.0),
    (66, 24, 3, "softmax", True, 12, 12, 2, True, 1.0), (5, 96, 20, "sigmoid", True, 32, 5, 2, False, 1.0),
    (11, 63, 40, "softmax", False, 63, 41, 2, True, 1.0),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", ["plain", "ties", "masked", "far"])
@pytest.mark.parametrize("t,e,k,score,bias,groups,tg,gt,renorm,scale", ROUTES)
def test_route(dtype, kind, t, e, k, score, bias, groups, tg, gt, renorm, scale):
    print(f"route {dtype} {kind} T={t} E={e} k={k} {score} bias={bias} groups={groups}/{tg}/{gt}", flush=True)
    g = np.random.default_rng(100 + t + e)
    l = g.standard_normal((t, e)) * 2
    if kind == "ties":
        l = np.round(l)
    if kind == "masked":
        l[g.random((t, e)) < 0.5] = -np.inf
        l[g.random((t, e)) < 0.1] = np.nan
        l[t // 2] = -np.inf
    if kind == "far":
        l = l * 200
    x = torch.from_numpy(l.astype(np.float32)).to(TYPES[dtype])
    b = None
    if bias:
        b = (0.1 * g.standard_normal(e)).astype(np.float32)
        if kind == "ties":
            b[:] = 0.25
    ids, w = qmm.route_experts(x.cuda(), k, score, None if b is None else torch.from_numpy(b).cuda(), groups, tg, gt,
                               renorm, scale)
    ri, rw = route_ref(x.double().numpy(), k, score, b, groups, tg, gt, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), ri)
    # 64-bit scores (a few 2^-52 off), one rounding to f32
    assert np.all(np.abs(f64(w) - rw) <= 2.0**-24 * (1 + 2.0**-20) * np.abs(rw) + 2.0**-150)


def test_route_infinite_logits_share_the_weight():
    x = torch.zeros((2, 8)).cuda()
    x[0, 3] = x[0, 6] = float("inf")
    ids, w = qmm.route_experts(x, 3, renormalize=False)
    assert ids[0].tolist() == [3, 6, 0] and w[0].tolist() == [0.5, 0.5, 0.0]
    assert ids[1].tolist() == [0, 1, 2] and w[1].tolist() == [0.125] * 3


# ---------------------------------------------------- the layer as a whole --

def moe_layer(fmt, wg, wu, wd, logits, x, k):
    ids, w = qmm.route_experts(logits, k, score="sigmoid", groups=4, top_groups=2, group_top=2)
    h = qmm.experts_glu(fmt, wg, wu, x, ids)
    return ids, w, h, qmm.experts_combine(fmt, wd, h, ids, w)


def layer_case(fmt, e, hidden, ffn, seed):
    out = []
    for i, (n, k) in enumerate(((ffn, hidden), (ffn, hidden), (hidden, ffn))):
        b, w, wa = weights_of(fmt, seed + i, e * n, k)
        out.append((torch.from_numpy(b.reshape(e, n, -1)).cuda(), w, wa))
    return out


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("t", [1, 6, 150])
def test_a_layer_of_experts(fmt, t):
    f, e, k, hidden, ffn = FMTS[fmt], 16, 4, 256, 512
    (wg, g64, ga64), (wu, u64, ua64), (wd, d64, da64) = layer_case(f, e, hidden, ffn, 110)
    x, xh = acts(115, (t, hidden), torch.float32)
    logits, lh = acts(116, (t, e), torch.float32)
    ids, w, h, y = moe_layer(f, wg, wu, wd, logits, x, k)
    ri, rw = route_ref(lh, k, "sigmoid", None, 4, 2, 2, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), ri)
    g, ga = product_ref(g64, ga64, e, ffn, ri, per_slot(xh, k))
    u, ua = product_ref(u64, ua64, e, ffn, ri, per_slot(xh, k))
    ag = act_ref(g, "silu")
    slack_h = 1.13 * BAR * ga * (np.abs(u) + BAR * ua) + np.abs(g) * BAR * ua + 2.0**-19 * np.abs(ag * u)
    p, pa = product_ref(d64, da64, e, hidden, ri, ag * u)
    pe, _ = product_ref(np.abs(d64), da64, e, hidden, ri, slack_h)  # what h's own error can become
    close(y, (p * rw[..., None]).sum(1), ((BAR * pa * 1.01 + pe) * rw[..., None]).sum(1) + 2.0**-22 * (pa * rw[..., None]).sum(1), "layer")


@pytest.mark.parametrize("t", [1, 6, 150])
def test_a_layer_on_streams_and_in_graphs(t):
    """The same values on another stream, from two streams at once, and from two captured graphs replayed
    side by side and with eager work between the replays."""
    f, e, k, hidden, ffn = qmm.Q4_K, 16, 4, 256, 512
    (wg, _, _), (wu, _, _), (wd, _, _) = layer_case(f, e, hidden, ffn, 120)
    xs = [acts(125 + i, (t, hidden), torch.bfloat16)[0] for i in range(2)]
    ls = [acts(127 + i, (t, e), torch.float32)[0] for i in range(2)]
    want = [moe_layer(f, wg, wu, wd, l, x, k)[3].clone() for l, x in zip(ls, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s, l, x in zip(streams, ls, xs):
            with torch.cuda.stream(s):
                got.append(moe_layer(f, wg, wu, wd, l, x, k)[3])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    # a stream given as an argument
    s = streams[0]
    ids, w = qmm.route_experts(ls[0], k, score="sigmoid", groups=4, top_groups=2, group_top=2, stream=s)
    h = qmm.experts_glu(f, wg, wu, xs[0], ids, stream=s)
    y = qmm.experts_combine(f, wd, h, ids, w, stream=s)
    s.synchronize()
    assert torch.equal(y, want[0])
    graphs, outs = [], []
    for s, l, x in zip(streams, ls, xs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(moe_layer(f, wg, wu, wd, l, x, k)[3])
        graphs.append(g)
    for i in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = moe_layer(f, wg, wu, wd, ls[i % 2], xs[i % 2], k)[3]
        torch.cuda.synchronize()
        assert torch.equal(eager, want[i % 2])
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fmt", ["Q8_0", "Q4_K"])
@pytest.mark.parametrize("t", [3, 40, 420, 2100])
def test_values_depend_on_their_own_row_alone(fmt, dtype, t):
    """Runs again, and with the tokens in another order, give the same bits: the order in which the sort's
    atomics place an expert's pairs, and with it their tile, does not show."""
    f, e, n, k, kk = FMTS[fmt], 5, 70, 3, 1024
    b, _, _ = weights_of(f, 140, e * n, kk)
    wd = torch.from_numpy(b.reshape(e, n, -1)).cuda()
    x, _ = acts(141, (t, kk), TYPES[dtype])
    ids = torch.from_numpy(choose(142, t, e, k, "twice")).cuda()
    g = torch.rand((t, k)).cuda()
    h = qmm.experts_glu(f, wd, wd, x, ids)
    y = qmm.experts_combine(f, wd, acts(143, (t, k, kk), TYPES[dtype])[0], ids, g)
    perm = torch.from_numpy(np.random.default_rng(144).permutation(t)).cuda()
    for _ in range(3):
        assert torch.equal(qmm.experts_glu(f, wd, wd, x, ids), h)
        assert torch.equal(qmm.experts_glu(f, wd, wd, x[perm].contiguous(), ids[perm].contiguous()), h[perm])
        hh = acts(143, (t, k, kk), TYPES[dtype])[0][perm].contiguous()
        assert torch.equal(qmm.experts_combine(f, wd, hh, ids[perm].contiguous(), g[perm].contiguous()), y[perm])


def test_given_outputs_and_refusals():
    f, e, n, k, t = qmm.Q4_0, 4, 24, 64, 3
    b, w, wa = weights_of(f, 130, e * n, k)
    wd = torch.from_numpy(b.reshape(e, n, -1)).cuda()
    x, _ = acts(131, (t, k), torch.float16)
    ids = torch.from_numpy(choose(132, t, e, 2, "any")).cuda()
    y = torch.full((t + 2, 2, n), 7.0, dtype=torch.float16).cuda()
    out = qmm.experts_matmul(f, wd, x, ids, y=y[:t])
    assert out.data_ptr() == y.data_ptr() and (y[t:] == 7).all()
    assert torch.equal(out, qmm.experts_matmul(f, wd, x, ids))
    with pytest.raises(TypeError):
        qmm.experts_matmul(f, wd, x.double(), ids)
    with pytest.raises(TypeError):
        qmm.experts_matmul(f, wd, x, ids.long())
    with pytest.raises(ValueError):
        qmm.experts_matmul(f, wd, x[:2], ids)
    with pytest.raises(ValueError):
        qmm.experts_matmul(f, wd, x[:, :32].contiguous(), ids)
    with pytest.raises(ValueError):
        qmm.experts_matmul(f, wd, x.t().contiguous().t(), ids)
    with pytest.raises(TypeError):
        qmm.experts_matmul(f, wd, x, ids, y=y[:t].float())
    with pytest.raises(qmm.QmmError):  # x not 16-byte aligned
        qmm.experts_matmul(f, wd, torch.zeros(t * k + 1, dtype=torch.float16).cuda()[1:].view(t, k), ids)
    with pytest.raises(ValueError):
        qmm.experts_glu(f, wd, wd[:, :8].contiguous(), x, ids)
    with pytest.raises(ValueError):
        qmm.experts_combine(f, wd, torch.zeros((t, 2, k)).cuda(), ids, torch.zeros((t, 3)).cuda())
    with pytest.raises(ValueError):
        qmm.experts_matmul(f, wd, x, ids.cpu())
    q, s, z, _ = w4_case(133, 8, 64, 32, True, torch.float16)
    xx = torch.zeros((2, 64)).cuda()
    with pytest.raises(ValueError):
        qmm.w4_matmul(q, s[:4], xx)
    with pytest.raises(ValueError):
        qmm.w4_matmul(q, s, xx, zeros=z[:, :1].contiguous())
    with pytest.raises(ValueError):
        qmm.w4_matmul(q, s, torch.zeros((2, 96)).cuda())
    with pytest.raises(qmm.QmmError):  # groups of 16
        qmm.w4_matmul(q, torch.zeros((8, 4)).cuda(), xx)
    with pytest.raises(ValueError):
        qmm.route_experts(torch.zeros((2, 8)).cuda(), 9)
    with pytest.raises(qmm.QmmError):
        qmm.route_experts(torch.zeros((2, 8)).cuda(), 2, groups=3)
    with pytest.raises(ValueError):
        qmm.route_experts(torch.zeros((2, 8)).cuda(), 2, score="relu")
    with pytest.raises(ValueError):
        qmm.route_experts(torch.zeros((2, 8)).cuda(), 2, bias=torch.zeros(9).cuda())


def test_more_pairs_than_the_sort_keeps_in_registers():
    """17000 pairs (16384 stay in registers), then 20 times that, some without an expert."""
    f, e, n, k, kk = qmm.Q8_0, 7, 33, 4, 64
    b, w, wa = weights_of(f, 150, e * n, kk)
    wd = torch.from_numpy(b.reshape(e, n, -1)).cuda()
    for t in (4096, 4250, 85000):
        ids_h = choose(151 + t, t, e, k, "twice")
        x, xh = acts(152 + t, (t, kk), torch.bfloat16)
        y = qmm.experts_matmul(f, wd, x, torch.from_numpy(ids_h).cuda())
        step = max(1, t // 3000)
        ref, a = product_ref(w, wa, e, n, ids_h[::step], per_slot(xh[::step], k))
        close(y[::step], ref, BAR * a, f"{t} tokens")


# ------------------------------------------- the kernels of larger calls --
#
# Which kernel runs depends on the number of pairs, the pairs per expert and
# the tiles of outputs: one pair per workgroup up to 48 pairs; 16, 32 or 64
# rows per workgroup up to 1024 pairs where there are few tiles; else tiles of
# 32, 64 or 128 rows.

def skewed(seed, t, e, k):
    """Experts with very different numbers of pairs, the last one without any."""
    g = np.random.default_rng(seed)
    return np.minimum((g.random((t, k)) ** 2 * (e - 1)).astype(np.int32), e - 2)


def products_case(fmt, dtype, t, e, k, n, kk, ids_h, ops, seed):
    f, dt = FMTS[fmt], TYPES[dtype]
    b, w, wa = weights_of(f, seed, e * n, kk)
    wd = torch.from_numpy(b.reshape(e, n, -1)).cuda()
    ids = torch.from_numpy(ids_h).cuda()
    x, xh = acts(seed + 1, (t, kk), dt)
    y, a = product_ref(w, wa, e, n, ids_h, per_slot(xh, k))
    if "run" in ops:
        close(qmm.experts_matmul(f, wd, x, ids), y, BAR * a, "experts_matmul")
    if "glu" in ops:  # the same matrix as gate and up
        ag = act_ref(y, "silu")
        slack = 1.13 * BAR * a * (np.abs(y) + BAR * a) + np.abs(y) * BAR * a + 2.0**-20 * np.abs(ag * y)
        close(qmm.experts_glu(f, wd, wd, x, ids), ag * y, slack, "experts_glu")
    if "combine" in ops:
        h, hh = acts(seed + 2, (t, k, kk), dt)
        y, a = product_ref(w, wa, e, n, ids_h, hh)
        g = np.random.default_rng(seed + 3).random((t, k)).astype(np.float32)
        gd = g.astype(np.float64)[:, :, None]
        close(qmm.experts_combine(f, wd, h, ids, torch.from_numpy(g).cuda()), (y * gd).sum(1), BAR * (a * gd).sum(1), "combine")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("t,e,k,n,mult,ops", [
    (1100, 6, 1, 70, 3, ("run", "glu", "combine")), (1400, 5, 1, 1300, 1, ("run", "glu")), (750, 9, 4, 1290, 2, ("run",)),
    (520, 40, 3, 136, 5, ("run", "combine")), (1025, 2, 1, 33, 6, ("glu", "combine")),
])
def test_tiles_of_every_size(fmt, dtype, t, e, k, n, mult, ops):
    print(f"tiles {fmt} {dtype} T={t} E={e} k={k} N={n} mult={mult}", flush=True)
    products_case(fmt, dtype, t, e, k, n, k_of(FMTS[fmt], mult), skewed(160 + t, t, e, k), ops, 161 + t)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("t,e,k,n,mult", [(60, 16, 4, 50, 2), (100, 8, 2, 33, 5), (70, 1, 1, 97, 3), (256, 4, 4, 40, 1), (49, 64, 1, 130, 6)])
def test_rows_of_every_count(fmt, dtype, t, e, k, n, mult):
    print(f"rows {fmt} {dtype} T={t} E={e} k={k} N={n} mult={mult}", flush=True)
    ids = choose(170 + t, t, e, k, "twice" if t != 256 else "any")
    products_case(fmt, dtype, t, e, k, n, k_of(FMTS[fmt], mult), ids, ("run", "glu", "combine"), 171 + t)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,n,k,group,zeros,sdtype", [
    (49, 33, 96, 32, True, "f16"), (50, 130, 384, 128, False, "f32"), (64, 61, 1056, 96, True, "bf16"), (65, 40, 640, 64, False, "f16"),
    (16, 1200, 4096, 128, True, "f16"), (31, 1200, 4096, 64, False, "f32"), (48, 1300, 4096, 32, True, "bf16"),
    (1100, 1300, 96, 32, True, "f16"), (1500, 1300, 384, 128, False, "bf16"), (3000, 1290, 160, 32, False, "f32"),
    (3001, 1300, 256, 256, True, "f32"), (1537, 1030, 288, 96, True, "f16"),
])
def test_w4_rows_and_tiles(dtype, m, n, k, group, zeros, sdtype):
    print(f"w4 {dtype} M={m} N={n} K={k} G={group} zeros={zeros} {sdtype}", flush=True)
    q, s, z, w = w4_case(180 + m, n, k, group, zeros, TYPES[sdtype])
    x, xh = acts(181 + m, (m, k), TYPES[dtype])
    close(qmm.w4_matmul(q, s, x, zeros=z), xh @ w.T, BAR * (np.abs(xh) @ np.abs(w).T), "w4")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMTS) + ["W4"])
@pytest.mark.parametrize("m", [1, 20, 60, 1100])
def test_long_rows(fmt, dtype, m):
    """K = 33024: more than the preparation keeps in registers, several parts of a wave's share of a row.
    A chain of f32 additions has one per 32 products (inside which a matrix product adds 32 in at most 32
    steps) and 32 more at most to join waves and parts: each is off by at most 2^-24 of A."""
    k, n = 33024, 9
    x, xh = acts(190 + m, (m, k), TYPES[dtype])
    if fmt == "W4":
        q, s, z, w = w4_case(191, n, k, 128, True, torch.float16)
        got, wa = qmm.w4_matmul(q, s, x, zeros=z), np.abs(w)
    else:
        b, w, wa = weights_of(FMTS[fmt], 192, n, k)
        got = qmm.experts_matmul(FMTS[fmt], torch.from_numpy(b.reshape(1, n, -1)).cuda(), x,
                                 torch.zeros((m, 1), dtype=torch.int32).cuda())[:, 0]
    close(got, xh @ w.T, (k / 32 + 64) * 2.0**-24 * (np.abs(xh) @ wa.T), "long rows")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", list(FMTS))
def test_wide_ranges_and_non_finite_rows_in_tiles(fmt, dtype):
    k, n, m = 512, 40, 1200
    x = torch.from_numpy(np.tile(value_rows(k), (m // 24, 1))).to(TYPES[dtype])
    bad = {25: float("nan"), 500: float("inf"), m - 1: float("-inf")}
    for r, v in bad.items():
        x[r, (37 * r) % k] = v
    b, w, wa = weights_of(FMTS[fmt], 200, n, k)
    y = qmm.experts_matmul(FMTS[fmt], torch.from_numpy(b.reshape(1, n, -1)).cuda(), x.cuda(),
                           torch.zeros((m, 1), dtype=torch.int32).cuda())[:, 0]
    for r in bad:
        assert not torch.isfinite(y[r]).any()
    good = [r for r in range(m) if r not in bad]
    xh = x.double().numpy()[good]
    with np.errstate(over="ignore"):
        close(y[good], xh @ w.T, BAR * (np.abs(xh) @ wa.T) + 2.0**-126 * k * wa.max(), "finite rows")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m", [1, 60, 1500])
def test_an_outlier_whose_weights_are_zero(dtype, m):
    """Values far below their row's largest: off by 2^-22 of themselves or 2^-40 of that one, as documented."""
    k, n = 256, 1024
    q, s, z, w = w4_case(210, n, k, 64, False, torch.float32)
    q[:, 50] = 0x88  # elements 100 and 101: zero weights
    w = w.copy()
    w[:, 100:102] = 0
    x, _ = acts(211, (m, k), TYPES[dtype])
    big = 60000.0 if dtype == "f16" else 2.0**24
    x[:, 100] = big
    x[:, 7] *= 2.0**-12
    xh = f64(x)
    aw = np.abs(w)
    lost = np.maximum(2.0**-22 * np.abs(xh), 2.0**-40 * big) if dtype != "f16" else 0 * xh
    close(qmm.w4_matmul(q, s, x), xh @ w.T, BAR * (np.abs(xh) @ aw.T) + lost @ aw.T, "outlier")


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("m", [2, 60, 1100])
def test_half_precision_below_its_normal_range(fmt, m):
    k, n = 256, 30
    x, xh = acts(215, (m, k), torch.float16, 2.0**-17)  # most values below 2^-14, kept exactly
    b, w, wa = weights_of(FMTS[fmt], 216, n, k)
    ids = torch.zeros((m, 1), dtype=torch.int32).cuda()
    got = qmm.experts_matmul(FMTS[fmt], torch.from_numpy(b.reshape(1, n, -1)).cuda(), x, ids)[:, 0]
    close(got, xh @ w.T, BAR * (np.abs(xh) @ wa.T), "subnormal rows")


@pytest.mark.parametrize("fmt", ["Q8_0", "Q4_K", "Q6_K"])
@pytest.mark.parametrize("t", [1, 60, 500])
def test_a_huge_slot_of_weight_zero_leaves_the_others(fmt, t):
    f, e, n, k, kk = FMTS[fmt], 4, 48, 3, 512
    b, w, wa = weights_of(f, 220, e * n, kk)
    h, _ = acts(221, (t, k, kk), torch.float32)
    h[:, 1] *= 1e25
    g = np.random.default_rng(222).random((t, k)).astype(np.float32)
    g[:, 1] = 0
    ids_h = choose(223, t, e, k, "any")
    y, a = product_ref(w, wa, e, n, ids_h, f64(h))
    gd = g.astype(np.float64)[:, :, None]
    got = qmm.experts_combine(f, torch.from_numpy(b.reshape(e, n, -1)).cuda(), h, torch.from_numpy(ids_h).cuda(), torch.from_numpy(g).cuda())
    close(got, (y * gd).sum(1), BAR * (a * gd).sum(1), "combine")


@pytest.mark.parametrize("m", [1, 60, 1500])
def test_w4_in_graphs_replayed_side_by_side(m):
    k, n = 512, 1030
    q, s, z, _ = w4_case(230, n, k, 128, True, torch.float16)
    xs = [acts(231 + i, (m, k), torch.bfloat16)[0] for i in range(2)]
    want = [qmm.w4_matmul(q, s, x, zeros=z) for x in xs]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for x, st in zip(xs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(qmm.w4_matmul(q, s, x, zeros=z))
        graphs.append(g)
    for i in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        eager = qmm.w4_matmul(q, s, xs[i % 2], zeros=z)
        torch.cuda.synchronize()
        assert torch.equal(eager, want[i % 2])
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("m,n", [(540000, 2), (540000, 16), (70000, 3)])
def test_w4_past_32_bit_offsets(m, n):
    """540000 x 4096 activations: more than 2^31 values and 2^32 bytes, in x and in the workspace."""
    k = 4096 if m > 500000 else 64
    q, s, z, w = w4_case(240, n, k, k, True, torch.float16)
    x = torch.empty((m, k), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(241))
    y = qmm.w4_matmul(q, s, x, zeros=z)
    at = torch.tensor([0, 1, 63, 64, m // 2 - 1, m // 2, m - 65, m - 2, m - 1])
    xh = f64(x[at.cuda()])
    close(y[at.cuda()], xh @ w.T, BAR * (np.abs(xh) @ np.abs(w).T), "w4")


@pytest.mark.parametrize("t", [1, 30, 100, 1100])
def test_experts_past_32_bit_offsets(t):
    """64 x 33000 x 2048 in Q8_0: 4.6e9 bytes, the last expert's last rows past 2^32; few of them not zero."""
    f, e, n, k = qmm.Q8_0, 64, 33000, 2048
    b, w, wa = weights_of(f, 250, 40, k)
    wd = torch.zeros((e, n, b.shape[1]), dtype=torch.uint8, device="cuda")
    wd[-1, -40:] = torch.from_numpy(b).cuda()
    x, xh = acts(251, (t, k), torch.float16)
    ids = torch.full((t, 1), e - 1, dtype=torch.int32).cuda()
    y = qmm.experts_matmul(f, wd, x, ids)[:, 0]
    close(y[:, -40:], xh @ w.T, BAR * (np.abs(xh) @ wa.T), "last rows")
    assert (y[:, :-40] == 0).all()
    h = qmm.experts_glu(f, wd, wd, x, ids)[:, 0]
    assert (h[:, :-40] == 0).all() and (h[:, -40:] != 0).any()
