"""Argument checks of the cache and attention calls on the host: every refusal
comes before any HIP call, with its status code."""
import ctypes

import pytest

import block_quantized_matmul_gguf_amd as qmm

MB = 1 << 20
K, V, TABLE, STARTS, LENGTHS, X, Y, OUT, WS = (0x10000000 + i * 64 * MB for i in range(9))  # never read or written
BASE = dict(format_k=qmm.Q8_0, format_v=qmm.Q4_0, pages=4, page_size=64, heads=2, dim=64, k=K, v=V, batch=2, table_width=3,
            table=TABLE, starts=STARTS, lengths=LENGTHS)


def call(what, T=5, type=0, x=X, y=Y, xs=None, ys=None, q_heads=4, scale=0.1, causal=1, window=0, softcap=0.0, max_length=0,
         out=OUT, lse=None, ws=WS, ws_bytes=32 * MB, null=False, **kw):
    f = {**BASE, **kw}
    c = qmm.CacheStruct(*(f[n] for n, _ in qmm.CacheStruct._fields_))
    c = None if null else c
    lib, row = qmm.lib(), f["heads"] * f["dim"]
    if what == "store":
        return lib.qmatmul_cache_store(c, T, type, x, row if xs is None else xs, y, row if ys is None else ys, None)
    if what == "load":
        return lib.qmatmul_cache_load(c, T, type, x, y, None)
    xs = q_heads * f["dim"] if xs is None else xs
    return lib.qmatmul_cache_attention(c, T, q_heads, type, x, xs, scale, causal, window, softcap, max_length, out, lse, ws,
                                       ws_bytes, None)


SHARED = [
    (dict(T=0), qmm.OK), (dict(T=0, k=None, x=None), qmm.OK), (dict(batch=0), qmm.OK),
    (dict(null=True), qmm.EINVAL), (dict(format_k=qmm.Q5_0), qmm.EUNSUPPORTED), (dict(format_v=qmm.Q4_K), qmm.EUNSUPPORTED),
    (dict(type=3), qmm.EUNSUPPORTED), (dict(type=-1), qmm.EUNSUPPORTED), (dict(dim=32), qmm.EUNSUPPORTED),
    (dict(dim=80), qmm.EUNSUPPORTED), (dict(dim=512), qmm.EUNSUPPORTED), (dict(dim=0), qmm.EUNSUPPORTED),
    (dict(heads=0), qmm.EINVAL), (dict(heads=1025), qmm.EINVAL), (dict(page_size=0), qmm.EINVAL), (dict(page_size=32), qmm.EINVAL),
    (dict(page_size=100), qmm.EINVAL), (dict(page_size=8256), qmm.EINVAL), (dict(page_size=-64), qmm.EINVAL),
    (dict(pages=-1), qmm.EINVAL), (dict(pages=1 << 31), qmm.EINVAL), (dict(batch=-1), qmm.EINVAL),
    (dict(batch=(1 << 20) + 1), qmm.EINVAL), (dict(batch=1 << 20, heads=4), qmm.EINVAL), (dict(table_width=-1), qmm.EINVAL), (dict(table_width=1 << 25), qmm.EINVAL),
    (dict(T=-1), qmm.EINVAL), (dict(T=(1 << 24) + 1), qmm.EINVAL), (dict(T=1 << 24, heads=16, q_heads=16), qmm.EINVAL),
    (dict(k=None), qmm.EINVAL), (dict(v=None), qmm.EINVAL), (dict(table=None), qmm.EINVAL), (dict(starts=None), qmm.EINVAL),
    (dict(lengths=None), qmm.EINVAL), (dict(k=K + 8), qmm.EINVAL), (dict(v=V + 4), qmm.EINVAL), (dict(table=TABLE + 2), qmm.EINVAL),
    (dict(starts=STARTS + 1), qmm.EINVAL), (dict(lengths=LENGTHS + 2), qmm.EINVAL), (dict(x=None), qmm.EINVAL),
    (dict(x=X + 8), qmm.EINVAL), (dict(type=2, x=X + 2), qmm.EINVAL),
]


@pytest.mark.parametrize("what", ["store", "load", "attention"])
@pytest.mark.parametrize("kw,status", SHARED, ids=str)
def test_refusals(what, kw, status):
    assert call(what, **kw) == status
    assert (qmm.last_error() == "") == (status == qmm.OK)


@pytest.mark.parametrize("kw", [dict(y=None), dict(y=Y + 4), dict(xs=127), dict(ys=64), dict(xs=129), dict(type=1, ys=132),
                                dict(xs=(1 << 31) + 4), dict(k=V + 4096, v=V), dict(x=K), dict(y=V), dict(x=K - 512), dict(table=K + 64),
                                dict(lengths=V + 64), dict(starts=K)], ids=str)
def test_store_refusals(kw):
    assert call("store", **kw) == qmm.EINVAL and qmm.last_error()


@pytest.mark.parametrize("kw", [dict(y=None), dict(y=Y + 4), dict(x=Y), dict(x=Y + 512), dict(x=K), dict(y=V + 16), dict(x=TABLE),
                                dict(y=STARTS)], ids=str)
def test_load_refusals(kw):
    assert call("load", **kw) == qmm.EINVAL and qmm.last_error()


@pytest.mark.parametrize("kw", [dict(q_heads=0), dict(q_heads=3), dict(q_heads=1026), dict(window=-1), dict(window=1 << 31),
                                dict(window=5, causal=0), dict(max_length=-1), dict(scale=float("nan")), dict(scale=float("inf")),
                                dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(softcap=1e-42),
                                dict(scale=3e38), dict(softcap=3e38), dict(out=None),
                                dict(out=OUT + 8), dict(lse=Y + 2), dict(xs=255), dict(xs=258), dict(out=X), dict(out=K),
                                dict(lse=X), dict(lse=OUT), dict(out=V + 256), dict(lse=LENGTHS), dict(T=1 << 18, q_heads=1024)], ids=str)
def test_attention_refusals(kw):
    assert call("attention", **kw) == qmm.EINVAL and qmm.last_error()


def workspace(T=5, q_heads=4, type=0, causal=1, window=0, max_length=0, **kw):
    f = {**BASE, "k": None, "v": None, "table": None, "starts": None, "lengths": None, **kw}
    c = qmm.CacheStruct(*(f[n] for n, _ in qmm.CacheStruct._fields_))
    return qmm.lib().qmatmul_cache_attention_workspace_bytes(c, T, q_heads, type, causal, window, max_length)


def test_workspace_sizes():
    for kw in (dict(), dict(T=0), dict(batch=0), dict(table_width=0), dict(table_width=4000), dict(table_width=4000, max_length=100),
               dict(T=5000, dim=128, type=2), dict(window=100)):
        assert workspace(**kw) >= 0
    for kw in (dict(q_heads=3), dict(dim=80), dict(type=9), dict(window=3, causal=0), dict(T=-1), dict(format_k=99), dict(max_length=-1)):
        assert workspace(**kw) == -1 and qmm.last_error()


def test_a_missing_workspace_is_refused():
    long = dict(T=2, table_width=2000, pages=4000)
    need = workspace(**long)
    if need:
        for kw in (dict(ws=None), dict(ws=WS + 8), dict(ws_bytes=need - 1), dict(ws=OUT), dict(ws=X), dict(ws=TABLE), dict(lse=WS)):
            assert call("attention", **{**long, "ws_bytes": need, **kw}) == qmm.EINVAL and qmm.last_error()


def test_bindings_refuse_wrong_tensors():
    torch = pytest.importorskip("torch")
    kc = torch.zeros((2, 1, 64, 68), dtype=torch.uint8)
    i = torch.zeros((1, 1), dtype=torch.int32)
    x = torch.zeros((1, 1, 64))
    with pytest.raises(ValueError, match="GPU"):
        qmm.cache_store(qmm.Q8_0, qmm.Q8_0, kc, kc, x, x, i, i[0], i[0])
    with pytest.raises(TypeError):
        qmm.cache_load(qmm.Q8_0, qmm.Q8_0, [1], kc, i, i[0], i[0], tokens=1)
    with pytest.raises(ValueError, match="GPU"):
        qmm.cache_attention(qmm.Q8_0, qmm.Q8_0, kc, kc, x, i, i[0], i[0])


def test_the_struct_has_the_headers_layout():
    assert ctypes.sizeof(qmm.CacheStruct) == 8 + 4 * 8 + 2 * 8 + 2 * 8 + 3 * 8
