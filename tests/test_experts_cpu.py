"""Argument checks of the mixture-of-experts calls and the 4-bit group products
on the host: every refusal comes before any HIP call, with its status code."""
import ctypes

import pytest

import block_quantized_matmul_gguf_amd as qmm

FAKE = 0x10000  # 16-byte aligned, never read: each call below is refused first
OUT = 0x20000


def route(logits=FAKE, type=0, T=4, E=16, bias=None, score=0, top_k=2, groups=1, top_groups=1, group_top=1,
          renormalize=1, scale=1.0, ids=OUT, weights=OUT):
    return qmm.lib().qmatmul_route_experts(logits, type, T, E, bias, score, top_k, groups, top_groups, group_top,
                                           renormalize, scale, ids, weights, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), qmm.OK), (dict(T=0, logits=None, ids=None, weights=None), qmm.OK),
    (dict(type=3), qmm.EUNSUPPORTED), (dict(score=2), qmm.EUNSUPPORTED),
    (dict(T=-1), qmm.EINVAL), (dict(T=(1 << 24) + 1), qmm.EINVAL), (dict(E=0), qmm.EINVAL), (dict(E=1025), qmm.EINVAL),
    (dict(top_k=0), qmm.EINVAL), (dict(top_k=17), qmm.EINVAL), (dict(E=128, top_k=65), qmm.EINVAL),
    (dict(groups=0), qmm.EINVAL), (dict(groups=3), qmm.EINVAL), (dict(E=130, groups=65), qmm.EINVAL),
    (dict(groups=4, top_groups=0), qmm.EINVAL), (dict(groups=4, top_groups=5), qmm.EINVAL),
    (dict(group_top=0), qmm.EINVAL), (dict(group_top=3), qmm.EINVAL),
    (dict(logits=None), qmm.EINVAL), (dict(ids=None), qmm.EINVAL), (dict(weights=None), qmm.EINVAL),
    (dict(logits=FAKE + 2), qmm.EINVAL), (dict(type=1, logits=FAKE + 1), qmm.EINVAL), (dict(ids=OUT + 2), qmm.EINVAL),
    (dict(weights=OUT + 2), qmm.EINVAL), (dict(bias=FAKE + 2), qmm.EINVAL),
])
def test_route_refusals(kw, status):
    assert route(**kw) == status
    assert (qmm.last_error() == "") == (status == qmm.OK)


def experts(product, format=qmm.Q8_0, E=4, N=8, K=256, T=2, top_k=2, type=0, act=0, w=FAKE, w2=FAKE, x=FAKE, ids=FAKE,
            weights=FAKE, y=OUT, ws=None, ws_bytes=0):
    lib = qmm.lib()
    if product == "run":
        return lib.qmatmul_experts_run(format, E, N, K, T, top_k, type, 0, w, x, ids, y, ws, ws_bytes, None)
    if product == "glu":
        return lib.qmatmul_experts_glu(format, E, N, K, T, top_k, type, act, w, w2, x, ids, y, ws, ws_bytes, None)
    return lib.qmatmul_experts_combine(format, E, N, K, T, top_k, type, w, x, ids, weights, y, ws, ws_bytes, None)


@pytest.mark.parametrize("product", ["run", "glu", "combine"])
@pytest.mark.parametrize("kw,status", [
    (dict(T=0), qmm.OK), (dict(T=0, w=None, x=None, ids=None, y=None), qmm.OK),
    (dict(format=7), qmm.EUNSUPPORTED), (dict(format=qmm.Q8_K), qmm.EUNSUPPORTED), (dict(type=3), qmm.EUNSUPPORTED),
    (dict(K=40), qmm.EBLOCK), (dict(format=qmm.Q4_K, K=96), qmm.EBLOCK),
    (dict(E=0), qmm.EINVAL), (dict(E=1025), qmm.EINVAL), (dict(N=0), qmm.EINVAL), (dict(K=0), qmm.EINVAL),
    (dict(T=-1), qmm.EINVAL), (dict(top_k=0), qmm.EINVAL), (dict(top_k=65), qmm.EINVAL),
    (dict(T=1 << 24, top_k=2), qmm.EINVAL), (dict(N=1 << 31), qmm.EINVAL), (dict(K=1 << 21), qmm.EINVAL),
    (dict(w=None), qmm.EINVAL), (dict(x=None), qmm.EINVAL), (dict(ids=None), qmm.EINVAL), (dict(y=None), qmm.EINVAL),
    (dict(w=FAKE + 8), qmm.EINVAL), (dict(x=FAKE + 4), qmm.EINVAL), (dict(ids=FAKE + 2), qmm.EINVAL),
    (dict(y=OUT + 2), qmm.EINVAL), (dict(type=2, y=OUT + 1), qmm.EINVAL),
])
def test_experts_refusals(product, kw, status):
    assert experts(product, **kw) == status
    assert (qmm.last_error() == "") == (status == qmm.OK)


def test_glu_and_combine_refusals():
    assert experts("glu", w2=None) == qmm.EINVAL
    assert experts("glu", w2=FAKE + 8) == qmm.EINVAL
    assert experts("glu", act=2) == qmm.EUNSUPPORTED
    assert experts("combine", weights=None) == qmm.EINVAL
    assert experts("combine", weights=FAKE + 2) == qmm.EINVAL


def w4(N=8, K=256, M=2, group=64, type=0, scale_type=1, q=FAKE, scales=FAKE, zeros=None, x=FAKE, y=OUT, ws=None,
       ws_bytes=0):
    return qmm.lib().qmatmul_w4_run(N, K, M, group, type, scale_type, q, scales, zeros, x, y, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), qmm.OK), (dict(M=0, q=None, scales=None, x=None, y=None), qmm.OK),
    (dict(type=3), qmm.EUNSUPPORTED), (dict(scale_type=-1), qmm.EUNSUPPORTED),
    (dict(group=0), qmm.EBLOCK), (dict(group=48), qmm.EBLOCK), (dict(group=96), qmm.EBLOCK), (dict(K=40, group=40), qmm.EBLOCK),
    (dict(N=0), qmm.EINVAL), (dict(K=-32), qmm.EINVAL), (dict(M=-1), qmm.EINVAL), (dict(M=(1 << 24) + 1), qmm.EINVAL),
    (dict(N=1 << 31), qmm.EINVAL), (dict(K=1 << 21), qmm.EINVAL),
    (dict(q=None), qmm.EINVAL), (dict(scales=None), qmm.EINVAL), (dict(x=None), qmm.EINVAL), (dict(y=None), qmm.EINVAL),
    (dict(q=FAKE + 4), qmm.EINVAL), (dict(x=FAKE + 4), qmm.EINVAL), (dict(scales=FAKE + 1), qmm.EINVAL),
    (dict(scale_type=0, scales=FAKE + 2), qmm.EINVAL), (dict(y=OUT + 2), qmm.EINVAL),
])
def test_w4_refusals(kw, status):
    assert w4(**kw) == status
    assert (qmm.last_error() == "") == (status == qmm.OK)


def test_workspace_sizes():
    lib = qmm.lib()
    for product in (qmm.EXPERTS_RUN, qmm.EXPERTS_GLU, qmm.EXPERTS_COMBINE, qmm.EXPERTS_RUN_SLOTS):
        for t in (0, 1, 3, 40, 700, 5000):
            assert lib.qmatmul_experts_workspace_bytes(product, qmm.Q4_K, 64, 1024, 2048, t, 8, qmm.BF16) >= 0
        assert lib.qmatmul_experts_workspace_bytes(product, qmm.Q4_K, 64, 1024, 2047, 1, 8, qmm.BF16) == -1
        assert lib.qmatmul_experts_workspace_bytes(product, qmm.Q4_K, 0, 1024, 2048, 1, 8, qmm.BF16) == -1
    assert lib.qmatmul_experts_workspace_bytes(4, qmm.Q4_K, 64, 1024, 2048, 1, 8, qmm.BF16) == -1
    for m in (0, 1, 17, 64, 4000):
        assert lib.qmatmul_w4_workspace_bytes(1537, 1536, m, 32, qmm.F32) >= 0
    assert lib.qmatmul_w4_workspace_bytes(1537, 1536, 4, 48, qmm.F32) == -1


def test_a_missing_workspace_is_refused():
    # shapes that need scratch memory refuse a call without it, or with too little or a misaligned one
    lib = qmm.lib()
    seen = 0
    for product, code in (("run", qmm.EXPERTS_RUN), ("glu", qmm.EXPERTS_GLU), ("combine", qmm.EXPERTS_COMBINE)):
        for t in (40, 5000):
            shape = dict(E=64, N=1024, K=2048, T=t, top_k=8, type=qmm.BF16, format=qmm.Q4_K)
            need = lib.qmatmul_experts_workspace_bytes(code, qmm.Q4_K, 64, 1024, 2048, t, 8, qmm.BF16)
            if need == 0:
                continue
            seen += 1
            assert experts(product, **shape) == qmm.EINVAL
            assert experts(product, ws=0x40000, ws_bytes=need - 1, **shape) == qmm.EINVAL
            assert experts(product, ws=0x40008, ws_bytes=need, **shape) == qmm.EINVAL
    need = lib.qmatmul_w4_workspace_bytes(1024, 2048, 4000, 64, qmm.BF16)
    if need:
        assert w4(N=1024, K=2048, M=4000, type=qmm.BF16) == qmm.EINVAL


def test_bindings_refuse_wrong_tensors():
    torch = pytest.importorskip("torch")
    cpu = torch.zeros((4, 16))
    with pytest.raises(ValueError, match="GPU"):
        qmm.route_experts(cpu, 2)
    with pytest.raises(TypeError):
        qmm.route_experts([1.0], 2)
    with pytest.raises(ValueError, match="GPU"):
        qmm.w4_matmul(torch.zeros((8, 16), dtype=torch.uint8), torch.zeros((8, 1)), torch.zeros((2, 32)))
    with pytest.raises(ValueError, match="GPU"):
        qmm.experts_matmul(qmm.Q8_0, torch.zeros((2, 8, 34), dtype=torch.uint8), torch.zeros((2, 32)),
                           torch.zeros((2, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="act"):
        qmm.experts_glu(qmm.Q8_0, None, None, None, None, act="relu")


@pytest.mark.parametrize("n,k,m,group,fits", [
    (8, 16384, 1 << 22, 128, False), (8, 16384, (1 << 22) - 1, 128, True), (8, 4096, 1 << 24, 32, False),
    (8, 4096, (1 << 24) - 4, 32, True), (1 << 24, 64, 1 << 24, 64, False), (1 << 24, 64, 1 << 13, 64, True),
])
def test_launches_of_2_to_the_32_threads_are_refused_w4(n, k, m, group, fits):
    need = qmm.lib().qmatmul_w4_workspace_bytes(n, k, m, group, qmm.BF16)
    assert (need > 0) == fits
    if not fits:
        assert need == -1 and "large" in qmm.last_error()
        assert w4(N=n, K=k, M=m, group=group, type=qmm.BF16, ws=0x40000, ws_bytes=1 << 60) == qmm.EINVAL
        assert "large" in qmm.last_error()


@pytest.mark.parametrize("product,code", [("run", qmm.EXPERTS_RUN), ("glu", qmm.EXPERTS_GLU), ("combine", qmm.EXPERTS_COMBINE)])
@pytest.mark.parametrize("e,n,k,t,top_k,fits", [
    (1024, 1 << 21, 32, 2048, 1, False), (1024, 1 << 20, 32, 1024, 1, True), (4, 64, 16384, 1 << 22, 1, False),
    (4, 64, 8192, 1 << 21, 8, None), (4, 64, 2048, 1 << 23, 2, True),
])
def test_launches_of_2_to_the_32_threads_are_refused_experts(product, code, e, n, k, t, top_k, fits):
    if fits is None:  # a row per token fits (2^21), a row per pair (2^24) does not
        fits = product != "combine"
    need = qmm.lib().qmatmul_experts_workspace_bytes(code, qmm.Q8_0, e, n, k, t, top_k, qmm.F16)
    assert (need > 0) == fits
    if not fits:
        assert need == -1 and "large" in qmm.last_error()
        assert experts(product, E=e, N=n, K=k, T=t, top_k=top_k, type=qmm.F16, ws=0x40000, ws_bytes=1 << 60) == qmm.EINVAL
        assert "large" in qmm.last_error()
