"""A pool without pages and a table without columns (empty tensors, whose pointers
are null): nothing is stored, zeros are read back, rows see nothing."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_matmul_gguf_amd as qmm  # noqa: E402

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    qmm.lib()


# sequences, rows of each, heads of the cache, query heads to each
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fk,fv", [(qmm.Q8_0, qmm.Q4_0), (qmm.Q4_0, qmm.Q8_0)])
@pytest.mark.parametrize("count,rows,heads,per", [(1, 1, 1, 1), (3, 5, 2, 4), (70, 2, 2, 1), (4, 64, 8, 8)])
@pytest.mark.parametrize("pages,width", [(0, 4), (0, 40), (0, 0), (5, 0)])
@pytest.mark.parametrize("dim", [64, 128])
def test_no_pages_or_no_columns(pages, width, count, rows, heads, per, dim, fk, fv, dtype):
    print(f"empty {pages} {width} {count} {rows} {heads}x{per} {dim} {fk} {fv} {dtype}", flush=True)
    dt, t = TYPES[dtype], count * rows
    kc, vc = (torch.full((pages, heads, 64, qmm.row_bytes(f, dim)), 9, dtype=torch.uint8, device="cuda") for f in (fk, fv))
    table = torch.zeros((count, width), dtype=torch.int32, device="cuda")
    starts = torch.arange(0, t + 1, rows, dtype=torch.int32, device="cuda")
    lengths = torch.full((count,), rows + 100, dtype=torch.int32, device="cuda")
    x = torch.randn((t, heads, dim), device="cuda").to(dt)
    cache, batch = (fk, fv, kc, vc), (table, starts, lengths)
    qmm.cache_store(*cache, x, x, *batch)
    assert (kc == 9).all() and (vc == 9).all()
    for back in qmm.cache_load(*cache, *batch, tokens=t, dtype=dt):
        assert back.shape == x.shape and (back == 0).all()
    q = torch.randn((t, heads * per, dim), device="cuda").to(dt)
    for kw in (dict(), dict(causal=False), dict(window=7), dict(softcap=3.0)):
        lse = torch.zeros((t, heads * per), device="cuda")
        out = qmm.cache_attention(*cache, q, *batch, lse=lse, **kw)
        assert out.shape == q.shape and (out == 0).all() and torch.isneginf(lse).all(), kw
