"""Workspaces of the experts' calls and the 4-bit group products, on the host: sizes are there where a call
sorts or prepares, and a call without enough of it is refused."""
import pytest

import block_quantized_matmul_gguf_amd as qmm

from test_experts_cpu import experts, w4


@pytest.mark.parametrize("product,code", [("run", qmm.EXPERTS_RUN), ("glu", qmm.EXPERTS_GLU), ("combine", qmm.EXPERTS_COMBINE)])
@pytest.mark.parametrize("type", [qmm.F32, qmm.F16, qmm.BF16])
@pytest.mark.parametrize("t", [40, 500, 5000])
def test_what_a_call_of_many_pairs_needs(product, code, type, t):
    e, n, k, top = 64, 1024, 2048, 8
    need = qmm.lib().qmatmul_experts_workspace_bytes(code, qmm.Q4_K, e, n, k, t, top, type)
    pairs, size = t * top, 4 if type == qmm.F32 else 2
    least = pairs * 4 + (pairs if code == qmm.EXPERTS_COMBINE else t) * k * size  # order and activations
    if code == qmm.EXPERTS_COMBINE:
        least += pairs * n * 4  # products in f32
    assert need >= least
    shape = dict(E=e, N=n, K=k, T=t, top_k=top, type=type, format=qmm.Q4_K)
    for ws, have in ((None, 0), (None, need), (0x40000, 0), (0x40000, need - 1), (0x40008, need)):
        assert experts(product, ws=ws, ws_bytes=have, **shape) == qmm.EINVAL
        assert "ws" in qmm.last_error()


@pytest.mark.parametrize("m", [60, 4000])
def test_what_a_4_bit_product_of_many_rows_needs(m):
    need = qmm.lib().qmatmul_w4_workspace_bytes(1024, 2048, m, 64, qmm.BF16)
    assert need >= m * 2048 * 2
    for ws, have in ((None, 0), (0x40000, need - 1), (0x40008, need)):
        assert w4(N=1024, K=2048, M=m, type=qmm.BF16, ws=ws, ws_bytes=have) == qmm.EINVAL
        assert "ws" in qmm.last_error()


def test_one_token_needs_none():
    for code in (qmm.EXPERTS_RUN, qmm.EXPERTS_GLU, qmm.EXPERTS_COMBINE, qmm.EXPERTS_RUN_SLOTS):
        assert qmm.lib().qmatmul_experts_workspace_bytes(code, qmm.Q4_K, 64, 1024, 2048, 1, 8, qmm.BF16) == 0
    assert qmm.lib().qmatmul_w4_workspace_bytes(1024, 2048, 1, 64, qmm.BF16) == 0
