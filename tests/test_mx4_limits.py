"""What the 4-bit products need and which kernels they take, by the library's own rules (no GPU here)."""
import ctypes

import pytest

import microscaling_quantized_convolution_amd as mq

BIG = (1 << 30) - 1


@pytest.mark.parametrize("m,n,k", [(0, 0, 0), (1, 1, 1), (8192, 8192, 8192), (BIG, BIG, BIG)])
def test_workspaces_hold_quantized_matrices_alone(m, n, k):
    """A product of two held matrices needs none; the layers hold their quantized inputs or gradients, codes
    and scales each from a multiple of 256 bytes."""
    L = mq.lib()
    part = lambda r, c: sum(-(-f(r, c) // 256) * 256 for f in (L.mq_mx4_codes_bytes, L.mq_mx4_scales_bytes))
    assert L.mq_mx4_matmul_workspace_bytes(m, n, k) == 0
    assert L.mq_mx4_linear_workspace_bytes(m, n, k) == part(m, k) == L.mq_mx4_gated_workspace_bytes(m, n, k)
    assert L.mq_mx4_linear_backward_workspace_bytes(m, n, k) == part(m, n) + part(n, m)
    assert L.mq_mx4_gated_backward_workspace_bytes(m, n, k) == 2 * (part(m, n) + part(n, m))
    empty, some = mq.mq_mx4(0, 64, 0, 0), mq.mq_mx4(8, 64, 0x20000, 0x30000)
    assert L.mq_mx4_matmul(empty, some, mq.mq_matrix(0, 8, 0, 8, mq.MQ_BF16), None, 0, ctypes.c_void_p(0)) == mq.MQ_OK
