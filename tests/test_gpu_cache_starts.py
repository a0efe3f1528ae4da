"""Starts that name rows outside the call's tensors: a sequence that has such rows
is left out as a whole, whatever the number of sequences and of pieces, and what
an earlier call left in the workspace does not matter.  And starts that begin far
behind row 0."""
import numpy as np
import pytest

import cache_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_matmul_gguf_amd as qmm  # noqa: E402
from attention_bounds import bounds  # noqa: E402
from test_gpu_attention import FMTS, TYPES, check, gpu, largest  # noqa: E402

CODES = {"f32": qmm.F32, "f16": qmm.F16, "bf16": qmm.BF16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    qmm.lib()


def batch_of(count, before, behind, rows, length):
    """starts of `count` sequences of `rows` rows each, the first `before` rows of which lie before row 0 and the last
    `behind` past the end (more than 2^20 rows: the first, and the last, sequence's alone); lengths; rows there are;
    sequences that are whole."""
    if before > 1 << 20 or behind > 1 << 20:
        starts = np.arange(-1, count, dtype=np.int64) * rows
        starts[0], starts[-1] = -before, behind
        t = int(starts[-2]) + 2
        return starts.astype(np.int32), [length] * count, t, list(range(1, count - 1))
    starts = np.arange(count + 1, dtype=np.int64) * rows - before
    t = int(starts[-1]) - behind
    whole = [s for s in range(count) if starts[s] >= 0 and starts[s + 1] <= t]
    return starts.astype(np.int32), [length] * count, t, whole


# sequences, rows before the first, rows behind the last, rows of each, tokens of each, pages in the table
CASES = [(2, 0, 3, 5, 700, 16), (2, 3, 0, 5, 700, 16), (4, 7, 1, 6, 130, 16), (2, 0, 3, 5, 700, 700 // 64 + 1), (2, 2, 0, 20, 40, 1),
         (70, 9, 5, 3, 600, 12), (130, 100, 80, 4, 70, 2), (130, 101, 81, 4, 70, 2), (70, 50, 50, 100, 120, 2),
         (4, 2**31, 2**31 - 1, 5, 700, 16), (70, 2**31, 2**31 - 1, 3, 600, 12), (80, 2**31 - 5, 2**31 - 9, 4, 70, 2),
         (3, -500, 0, 5, 700, 16), (70, -500, 4, 3, 600, 12), (70, -501, 30, 100, 120, 2)]


def make(case, fk="q8", fv="q4", heads=1, dim=64):
    count, before, behind, rows, length, width = case
    starts, lengths, t, whole = batch_of(count, before, behind, rows, length)
    c = ref.Cache(320, FMTS[fk], FMTS[fv], heads, dim, 64, lengths, width=width)
    return c, starts, t, whole


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention(case, dtype):
    print(f"starts {case} {dtype}", flush=True)
    c, starts, t, whole = make(case)
    dt, per, dim = TYPES[dtype], 2, c.dim
    q = torch.from_numpy(np.random.default_rng(1).standard_normal((t, per, dim)).astype(np.float32)).to(dt)
    qd, kc, vc, table, st, ln = q.cuda(), gpu(c.k_cache), gpu(c.v_cache), gpu(c.table), gpu(starts), gpu(c.lengths)
    out = torch.full((t, per, dim), 7.0, device="cuda", dtype=dt)
    lse = torch.full((t, per), 7.0, device="cuda")
    cache = qmm.CacheStruct(c.fmt_k, c.fmt_v, len(kc), c.page_size, c.heads, dim, kc.data_ptr(), vc.data_ptr(), len(ln),
                            table.shape[1], table.data_ptr(), st.data_ptr(), ln.data_ptr())
    need = qmm.lib().qmatmul_cache_attention_workspace_bytes(cache, t, per, CODES[dtype], 1, 0, 0)
    assert need >= 0
    ws = torch.full((need // 4 + 4,), 2, dtype=torch.int32, device="cuda")  # two pieces of nothing, as another call may leave it
    status = qmm.lib().qmatmul_cache_attention(cache, t, per, CODES[dtype], qd.data_ptr(), per * dim, dim ** -0.5, 1, 0, 0.0, 0,
                                               out.data_ptr(), lse.data_ptr(), ws.data_ptr(), need,
                                               torch.cuda.current_stream().cuda_stream)
    assert status == qmm.OK
    average = -(-t * per // len(ln))
    kernel = "many" if dtype != "f32" and average >= 192 and -(-average // 16) * len(ln) >= 512 else "rows"
    left = np.ones(t, dtype=bool)
    for s in whole:
        rows = slice(starts[s], starts[s + 1])
        left[rows] = False
        n, m = int(c.lengths[s]), int(starts[s + 1] - starts[s])
        o, l, big, top = ref.attention(q[rows].double().numpy(), c.kq[s], c.vq[s], np.arange(n - m, n), dim ** -0.5)
        tol, of_lse = bounds(kernel, dt, dim, n, big, top, largest(c.vq[s]), l)
        check(out[rows], o, tol, f"out of sequence {s}")
        check(lse[rows], l, of_lse, f"lse of sequence {s}")
    assert whole
    left = torch.from_numpy(left).cuda()
    assert (out[left] == 7).all() and (lse[left] == 7).all(), "rows of sequences that are left out"


@pytest.mark.parametrize("fk,fv", [("q8", "q4"), ("q4", "q8")])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_store_and_load(case, fk, fv):
    c, starts, t, whole = make(case, fk, fv, heads=2)
    rng = np.random.default_rng(2)
    k, v = (rng.standard_normal((t, 2, c.dim)).astype(np.float32) for _ in range(2))
    kc, vc = gpu(c.k_cache), gpu(c.v_cache)
    batch = gpu(c.table), gpu(starts), gpu(c.lengths)
    qmm.cache_store(c.fmt_k, c.fmt_v, kc, vc, gpu(k), gpu(v), *batch)
    back = [np.full((t, 2, c.dim), 7.0) for _ in range(2)]
    for s in whole:
        rows, m = slice(starts[s], starts[s + 1]), int(starts[s + 1] - starts[s])
        c.k[s][-m:], c.v[s][-m:] = k[rows], v[rows]
    c.write()
    for s in whole:
        rows, m = slice(starts[s], starts[s + 1]), int(starts[s + 1] - starts[s])
        back[0][rows], back[1][rows] = c.kq[s][-m:], c.vq[s][-m:]
    assert np.array_equal(kc.cpu().numpy(), c.k_cache) and np.array_equal(vc.cpu().numpy(), c.v_cache)
    got = [torch.full((t, 2, c.dim), 7.0, device="cuda") for _ in range(2)]
    qmm.cache_load(c.fmt_k, c.fmt_v, kc, vc, *batch, tokens=t, k=got[0], v=got[1])
    for g, b in zip(got, back):
        assert torch.equal(g.cpu(), torch.from_numpy(b).float())
