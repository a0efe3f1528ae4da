"""Outputs that overlap inputs, or each other, are refused on the host: workgroups write while others still
read, so such a call has no defined values."""
import pytest

import block_quantized_matmul_gguf_amd as qmm

from test_experts_cpu import experts, route, w4

FAR = 1 << 40  # every call below is refused before anything is read
W, W2, X, IDS, G, Y, WS = (FAR + i * (1 << 36) for i in range(7))
SHAPE = dict(format=qmm.Q8_0, E=4, N=64, K=256, T=200, top_k=2, type=qmm.BF16)
BYTES = dict(w=4 * 64 * 272, w2=4 * 64 * 272, ids=200 * 2 * 4, weights=200 * 2 * 4)
AT = dict(w=W, w2=W2, x=X, ids=IDS, weights=G)


def need(product):
    code = {"run": qmm.EXPERTS_RUN, "glu": qmm.EXPERTS_GLU, "combine": qmm.EXPERTS_COMBINE}[product]
    return qmm.lib().qmatmul_experts_workspace_bytes(code, qmm.Q8_0, 4, 64, 256, 200, 2, qmm.BF16)


def sizes(product):
    rows = 400 if product == "combine" else 200
    return dict(BYTES, x=rows * 256 * 2), (200 if product == "combine" else 400) * 64 * 2


@pytest.mark.parametrize("product,reads", [("run", ("w", "x", "ids")), ("glu", ("w", "w2", "x", "ids")),
                                           ("combine", ("w", "x", "ids", "weights"))])
def test_outputs_and_workspaces_of_products(product, reads):
    ws_bytes, (held, y_bytes) = need(product), sizes(product)
    assert ws_bytes > 0
    for name in reads:
        last = (AT[name] + held[name] - 1) // 16 * 16
        for at in (AT[name], last, AT[name] - y_bytes + 16):
            assert experts(product, **SHAPE, **AT, y=at, ws=WS, ws_bytes=ws_bytes) == qmm.EINVAL
            assert "overlap" in qmm.last_error(), (name, at)
        for at in (AT[name], last, AT[name] - ws_bytes + 16):
            assert experts(product, **SHAPE, **AT, y=Y, ws=at, ws_bytes=ws_bytes) == qmm.EINVAL
            assert "overlap" in qmm.last_error(), (name, at)
    for at in (Y, Y - ws_bytes + 16, Y + y_bytes - 16):
        assert experts(product, **SHAPE, **AT, y=Y, ws=at, ws_bytes=ws_bytes) == qmm.EINVAL
        assert "overlap" in qmm.last_error()


def test_outputs_and_workspaces_of_4_bit_products():
    n, k, m, group = 64, 256, 200, 64
    ws_bytes = qmm.lib().qmatmul_w4_workspace_bytes(n, k, m, group, qmm.BF16)
    args = dict(N=n, K=k, M=m, group=group, type=qmm.BF16, scale_type=qmm.F32, q=W, scales=G, zeros=IDS, x=X, ws=WS, ws_bytes=ws_bytes)
    assert ws_bytes > 0
    for at, size in ((W, n * k // 2), (G, n * 4 * 4), (IDS, n * 4), (X, m * k * 2), (WS, ws_bytes)):
        for y in (at, (at + size - 1) // 16 * 16, at - m * n * 2 + 16):
            assert w4(**args, y=y) == qmm.EINVAL
            assert "overlap" in qmm.last_error(), (at, y)
    args["ws"] = X + 16
    assert w4(**args, y=Y) == qmm.EINVAL and "overlap" in qmm.last_error()


@pytest.mark.parametrize("kw", [
    dict(ids=X), dict(ids=X + 4 * 16 * 4 - 4), dict(ids=X - 4 * 2 * 4 + 4), dict(weights=X), dict(ids=G), dict(weights=G + 60),
    dict(ids=Y, weights=Y), dict(ids=Y, weights=Y + 28), dict(ids=Y, weights=Y - 28),
])
def test_outputs_of_the_router(kw):
    args = dict(dict(logits=X, bias=G, ids=IDS, weights=WS), **kw)
    assert route(**args) == qmm.EINVAL
    assert "overlap" in qmm.last_error()
