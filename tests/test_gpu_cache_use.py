"""The cache and the attention over it as a server uses them: a layer from its
GGUF products to its output product, graphs that are replayed while sequences
grow, other streams, batches of many sequences, tensors past 32 bits.  The
tolerances are those of the attention's own tests."""
import numpy as np
import pytest

import cache_ref as ref
import oracle
import synth
from test_gpu_attention import FMTS, LOSS_P, TYPES, check, gpu, largest, run_case, slack, starts_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_matmul_gguf_amd as qmm  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    qmm.lib()


def pool(fk, fv, pages, heads, dim, page=64):
    return tuple(torch.zeros((pages, heads, page, qmm.row_bytes(f, dim)), dtype=torch.uint8, device="cuda") for f in (fk, fv))


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fk,fv", [("q8", "q8"), ("q8", "q4")])
def test_a_layer_over_a_prompt_and_single_tokens(fk, fv):
    """q, k and v products, store, attention, output product: a prompt of 37 tokens, then four tokens one by one
    (hidden size 576, 9 query heads on 3, dim 64)."""
    hidden, heads, per, dim = 576, 3, 3, 64
    fk, fv = FMTS[fk], FMTS[fv]
    shapes = [heads * per * dim, heads * dim, heads * dim]
    w = [oracle.quantize(qmm.Q8_0, synth.weights_f32(60 + i, n, hidden)) for i, n in enumerate(shapes)]
    wo = oracle.quantize(qmm.Q8_0, synth.weights_f32(70, hidden, heads * per * dim))
    wd, wod = [torch.from_numpy(b).cuda() for b in w], torch.from_numpy(wo).cuda()
    plans = [qmm.Plan(qmm.Q8_0, n, hidden, 64, qmm.MODE_F32ACT) for n in shapes]
    out_plan = qmm.Plan(qmm.Q8_0, hidden, heads * per * dim, 64, qmm.MODE_F32ACT)
    kc, vc = pool(fk, fv, 4, heads, dim)
    table = ints(2, 0)[None]
    keys, values = [], []
    length = 0
    for step, n in enumerate((37, 1, 1, 1, 30)):
        x = torch.from_numpy(synth.acts_f32(80 + step, n, hidden) * 4).cuda()
        q, k, v = qmm.run_group(plans, wd, x)
        length += n
        batch = table, ints(0, n), ints(length)
        qmm.cache_store(fk, fv, kc, vc, k.view(n, heads, dim), v.view(n, heads, dim), *batch)
        lse = torch.empty((n, heads * per), device="cuda")
        a = qmm.cache_attention(fk, fv, kc, vc, q.view(n, heads * per, dim), *batch, lse=lse)
        y = out_plan.run(wod, a.view(n, -1))
        keys.append(ref.values(*ref.quantize(fk, k.view(n, heads, dim).cpu().numpy())))
        values.append(ref.values(*ref.quantize(fv, v.view(n, heads, dim).cpu().numpy())))
        kk, vv = np.concatenate(keys), np.concatenate(values)
        o, l, big, top = ref.attention(q.view(n, heads * per, dim).cpu().double().numpy(), kk, vv, np.arange(length - n, length), dim ** -0.5)
        tol, e = slack(torch.float32, dim, length, big, top, largest(vv))
        check(a, o, tol, f"attention of step {step}")
        yr, mag = oracle.matmul_a(qmm.Q8_0, wo, hidden, heads * per * dim, a.view(n, -1).cpu().numpy())
        assert (np.abs(y.cpu().double().numpy() - yr) <= 1e-5 * mag).all()
    for p in plans + [out_plan]:
        p.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fk,fv,bound", [("q8", "q8", 0), ("q4", "q8", 4096)])
def test_graphs_replayed_while_sequences_grow(fk, fv, bound, dtype):
    """Store and attention of one token per sequence as two graphs over two caches, replayed in turn with inputs and
    lengths changed in place; with a table of 4096 positions the work is in pieces, so each has a workspace."""
    f, dt, heads, per, dim, page = (FMTS[fk], FMTS[fv]), TYPES[dtype], 2, 4, 128, 64
    width, first = 64, [700, 60]
    sides = []
    for side in range(2):
        g = torch.Generator(device="cuda").manual_seed(side)
        caches = pool(*f, 2 * width, heads, dim, page)
        table = torch.randperm(2 * width, device="cuda", generator=g).to(torch.int32).view(2, width)
        k, v = (torch.randn((sum(first), heads, dim), device="cuda", generator=g).to(dt) for _ in range(2))
        qmm.cache_store(*f, *caches, k, v, table, ints(0, first[0], sum(first)), ints(*first))
        s = dict(caches=caches, mirror=tuple(c.clone() for c in caches), table=table, lengths=ints(*first), starts=ints(0, 1, 2), g=g)
        s["q"] = torch.zeros((2, heads * per, dim), device="cuda", dtype=dt)
        s["k"], s["v"] = (torch.zeros((2, heads, dim), device="cuda", dtype=dt) for _ in range(2))
        sides.append(s)

    def step(s, caches):
        qmm.cache_store(*f, *caches, s["k"], s["v"], s["table"], s["starts"], s["lengths"])
        return qmm.cache_attention(*f, *caches, s["q"], s["table"], s["starts"], s["lengths"], max_length=bound)

    for s in sides:
        step(s, tuple(c.clone() for c in s["caches"]))  # once eagerly
    torch.cuda.synchronize()
    for s in sides:
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"]):
            s["out"] = step(s, s["caches"])
    for turn in range(6):
        for s in sides:
            s["lengths"] += 1
            for name in "qkv":
                s[name].copy_(torch.randn(s[name].shape, device="cuda", generator=s["g"]).to(dt))
        for s in sides:
            s["graph"].replay()
        for s in sides:
            want = step(s, s["mirror"])
            assert torch.equal(s["out"], want), f"turn {turn}"
            assert all(torch.equal(a, b) for a, b in zip(s["caches"], s["mirror"])), f"turn {turn}"
        torch.cuda.synchronize()


def test_calls_on_other_streams():
    """Two streams over one cache at once, each waiting for the work that made its inputs."""
    heads, per, dim, n = 2, 4, 128, 6000
    c = ref.Cache(5, 8, 8, heads, dim, 128, [n])
    args = 8, 8, gpu(c.k_cache), gpu(c.v_cache)
    batch = gpu(c.table), ints(0, 2), gpu(c.lengths)
    q = [torch.randn((2, heads * per, dim), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    want = [qmm.cache_attention(*args, x, *batch) for x in q]
    back = qmm.cache_load(*args, batch[0], ints(0, n), batch[2], tokens=n)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i].append(qmm.cache_attention(*args, q[i], *batch, stream=s))
    loaded = qmm.cache_load(*args, batch[0], ints(0, n), batch[2], tokens=n, stream=streams[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])
    assert all(torch.equal(a, b) for a, b in zip(loaded, back))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("count", [65, 700, 4500])
def test_many_sequences(count, dtype):
    """More sequences than a wave has lanes, and than 64 of those; some with no rows, some with no tokens."""
    dt, heads, per, dim, page = TYPES[dtype], 1, 2, 64, 64
    rng = np.random.default_rng(count)
    lengths = rng.integers(0, 100, count)
    new = np.minimum(lengths, rng.integers(0, 4, count))
    c = ref.Cache(3, 8, 2, heads, dim, page, list(lengths), width=2)
    st = starts_of(new)
    t = int(st[-1])
    k = torch.from_numpy(rng.standard_normal((t, heads, dim)).astype(np.float32)).to(dt)
    kh = k.float().numpy()
    kc, vc = gpu(c.k_cache), gpu(c.v_cache)
    batch = gpu(c.table), gpu(st), gpu(c.lengths)
    qmm.cache_store(8, 2, kc, vc, k.cuda(), k.cuda(), *batch)
    for s, n in enumerate(lengths):
        c.k[s][n - new[s]:] = c.v[s][n - new[s]:] = kh[st[s]:st[s + 1]]
    c.write()
    assert np.array_equal(kc.cpu().numpy(), c.k_cache) and np.array_equal(vc.cpu().numpy(), c.v_cache)
    q = torch.from_numpy(rng.standard_normal((t, heads * per, dim)).astype(np.float32)).to(dt)
    out = qmm.cache_attention(8, 2, kc, vc, q.cuda(), *batch)
    want, tol = np.zeros(out.shape), np.zeros(out.shape)
    for s, n in enumerate(lengths):
        if new[s]:
            rows = slice(st[s], st[s + 1])
            o, _, big, top = ref.attention(q[rows].double().numpy(), c.kq[s], c.vq[s], np.arange(n - new[s], n), dim ** -0.5)
            want[rows], tol[rows] = o, slack(dt, dim, n, big, top, largest(c.vq[s]))[0]
    check(out, want, tol, "out")


# many rows of a sequence: every dim and type, tiles with few rows, pieces, windows, pages that are not there
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fk,fv", [("q8", "q8"), ("q4", "q4"), ("q4", "q8")])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("lengths,new,heads,per,kw", [
    ([900], [130], 1, 1, {}), ([2500, 140], [150, 140], 1, 2, {}), ([1300, 1, 700], [260, 1, 130], 1, 3, dict(window=200)),
    ([1100], [300], 2, 4, dict(causal=False)), ([3000], [129], 1, 1, dict(window=1000, softcap=10.0)), ([256], [256], 1, 1, {}),
])
def test_many_rows(lengths, new, heads, per, kw, dim, fk, fv, dtype):
    print(f"many rows {lengths} {new} {heads}x{per} {kw} {dim} {fk} {fv} {dtype}", flush=True)
    run_case(100 + dim, fk, fv, dtype, heads, per, dim, 128, lengths, new, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("new,per", [(1, 2), (200, 2)])
def test_pages_that_are_not_there(new, per, dtype):
    """Entries of the table that name no page, at the start, alone, in runs, at the end: their positions are not seen."""
    dt, heads, dim, page, n = TYPES[dtype], 1, 128, 64, 64 * 40 - 20
    c = ref.Cache(9, 8, 8, heads, dim, page, [n])
    gone = [0, 1, 5, 9, 10, 11, 12, 13, 14, 30, 38, 39]
    c.table[0, gone] = [-1, 10**6, -2**31, 2**31 - 1, -1, -1, 41, -1, -1, 100, -1, -1]
    seen = ~np.isin(np.arange(n) // page, gone)
    q = torch.from_numpy(np.random.default_rng(1).standard_normal((new, per, dim)).astype(np.float32)).to(dt)
    args = 8, 8, gpu(c.k_cache), gpu(c.v_cache), q.cuda(), gpu(c.table), ints(0, new), gpu(c.lengths)
    for window in (0, 300, 100):  # the last: rows that see only pages that are not there
        out = qmm.cache_attention(*args, window=window)
        o, l, big, top = ref.attention(q.double().numpy(), c.kq[0], c.vq[0], np.arange(n - new, n), dim ** -0.5, window=window, seen=seen)
        check(out, o, slack(dt, dim, n, big, top, largest(c.vq[0]))[0], f"window {window}")


def test_rows_past_2_to_the_31_values():
    """q, out and lse with more than 2^31 values, k and v with more than 2^32 bytes: the last sequences' rows."""
    heads, dim, page, each = 64, 256, 64, 64
    count = 2064  # sequences of 64 tokens: 132096 * 64 * 256 values
    t = count * each
    assert t * heads * dim > 1 << 31
    caches = pool(qmm.Q8_0, qmm.Q4_0, count, heads, dim, page)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((t, heads, dim), device="cuda", generator=g, dtype=torch.bfloat16)
    table = torch.randperm(count, device="cuda", generator=g).to(torch.int32).view(count, 1)
    starts = torch.arange(0, t + 1, each, device="cuda", dtype=torch.int32)
    lengths = torch.full((count,), each, device="cuda", dtype=torch.int32)
    qmm.cache_store(qmm.Q8_0, qmm.Q4_0, *caches, k, k, table, starts, lengths)
    gk, gv = qmm.cache_load(qmm.Q8_0, qmm.Q4_0, *caches, table, starts, lengths, tokens=t, dtype=torch.bfloat16)
    lse = torch.empty((t, heads), device="cuda")
    out = qmm.cache_attention(qmm.Q8_0, qmm.Q4_0, *caches, k, table, starts, lengths, lse=lse)
    for s in (0, 1000, count - 1):
        rows = slice(s * each, (s + 1) * each)
        x = k[rows].float().cpu().numpy()
        kk, vv = ref.values(*ref.quantize(8, x)), ref.values(*ref.quantize(2, x))
        for got, want in ((gk, kk), (gv, vv)):
            assert torch.equal(got[rows].cpu(), torch.from_numpy(want).to(torch.bfloat16))
        o, l, big, top = ref.attention(x.astype(np.float64), kk, vv, np.arange(each), dim ** -0.5)
        tol, e = slack(torch.bfloat16, dim, each, big, top, largest(vv))
        check(out[rows], o, tol, f"out of sequence {s}")
        check(lse[rows], l, 2 * e + 2.0**-19 + LOSS_P[torch.bfloat16], f"lse of sequence {s}")


def test_bindings_refuse_wrong_gpu_tensors():
    kc, vc = pool(8, 2, 3, 2, 64)
    i = ints(0)[None], ints(0, 1), ints(1)
    x = torch.zeros((1, 2, 64), device="cuda")
    good = lambda **kw: qmm.cache_store(*(kw.get(n, v) for n, v in zip("fgabxyts l".replace(" ", ""), (8, 2, kc, vc, x, x, *i))))  # noqa: E731
    good()
    for kw, err in ((dict(f=6), ValueError), (dict(g=12), ValueError), (dict(a=kc[:, :, :, :-2].contiguous()), ValueError),
                    (dict(b=kc), ValueError), (dict(a=kc[:, ::2]), ValueError), (dict(a=kc.int()), TypeError), (dict(x=x.double()), TypeError),
                    (dict(x=x[:, :1]), ValueError), (dict(y=x.half()), ValueError), (dict(x=x.cpu()), ValueError),
                    (dict(t=i[0].long()), TypeError), (dict(t=i[0][0]), ValueError), (dict(s=ints(0, 1, 2)), ValueError),
                    (dict(l=ints(1, 2)), ValueError), (dict(l=i[2].cpu()), ValueError), (dict(s=None), TypeError),
                    (dict(x=torch.zeros((1, 64, 2), device="cuda").transpose(1, 2)), ValueError)):
        with pytest.raises(err):
            good(**kw)
    with pytest.raises(ValueError):
        qmm.cache_load(8, 2, kc, vc, *i, tokens=-1)
    with pytest.raises(TypeError):
        qmm.cache_load(8, 2, kc, vc, *i, tokens=1, dtype=torch.float64)
    for kw in (dict(lse=torch.zeros((1, 3), device="cuda")), dict(out=torch.zeros((1, 2, 32), device="cuda"))):
        with pytest.raises(ValueError):
            qmm.cache_attention(8, 2, kc, vc, x, *i, **kw)
    with pytest.raises(qmm.QmmError):
        qmm.cache_attention(8, 2, kc, vc, torch.zeros((1, 3, 64), device="cuda"), *i)
    with pytest.raises(qmm.QmmError):  # a step of 66 halves is no multiple of 16 bytes
        y = torch.zeros((2, 132), device="cuda", dtype=torch.float16)[:, :128].view(2, 2, 64)
        qmm.cache_store(8, 2, kc, vc, y, y, ints(0)[None], ints(0, 2), ints(2))


def test_calls_without_tokens():
    kc, vc = pool(8, 8, 1, 1, 64)
    none = torch.zeros((0, 1, 64), device="cuda")
    i = ints(0)[None], ints(0, 0), ints(0)
    qmm.cache_store(8, 8, kc, vc, none, none, *i)
    k, v = qmm.cache_load(8, 8, kc, vc, *i, tokens=0)
    assert k.shape == v.shape == (0, 1, 64)
    assert qmm.cache_attention(8, 8, kc, vc, none, *i).shape == (0, 1, 64)
    out = torch.full((3, 1, 64), 7.0, device="cuda")  # a batch of no sequences: no row belongs to one
    qmm.cache_attention(8, 8, kc, vc, out.clone(), torch.zeros((0, 1), dtype=torch.int32, device="cuda"), ints(0), ints(1)[:0], out=out)
    assert (out == 7).all()
