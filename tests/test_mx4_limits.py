"""What the 4-bit products need and which kernels they take, by the library's own rules (no GPU here)."""
import ctypes

import pytest

import microscaling_quantized_convolution_amd as mq

BIG = (1 << 30) - 1
KINDS = ["rows", "64", "128 deep", "128", "256"]


def rule(name, *types):
    """A function of the library's own, which the launches ask too (csrc/mq_mx4.hpp)."""
    f = getattr(mq.lib(), name)
    f.restype, f.argtypes = ctypes.c_int, types
    return f


I, B = ctypes.c_int, ctypes.c_bool
matmul_kind = rule("_ZN2mq15mx4_matmul_kindEiiiib", I, I, I, I, B)
quantize_height = rule("_ZN2mq19mx4_quantize_heightEiiibb", I, I, I, B, B)


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


def test_kinds():
    """What the rule's comments give as measured takes the kernel that they name."""
    def kind(m, n, k, jobs=1, gated=False):
        return KINDS[matmul_kind(jobs, m, n, -(-k // 256), gated)]
    for size, name in (((16, 4096, 8192), "rows"), ((16, 4096, 16384), "rows"), ((256, 4096, 4096), "64"), ((512, 4096, 4096), "64"),
                       ((1024, 4096, 4096), "128 deep"), ((2048, 2048, 8192), "128 deep"), ((2048, 4096, 4096), "128"),
                       ((4096, 4096, 512), "128"), ((4096, 4096, 4096), "256"), ((8192, 8192, 4096), "256")):
        assert kind(*size) == name, size
    for m, n, gated, name in ((16, 8192, False, "rows"), (16, 8193, False, "64"), (4, 12288, False, "rows"),
                              (4, 12289, False, "64"), (1, 8192, True, "rows"), (1, 8193, True, "64"), (17, 16, False, "64")):
        assert kind(m, n, 4096, gated=gated) == name, (m, n, gated)
    assert kind(13, 4097, 300, jobs=2) == "64"
    assert kind(300, 2700, 1024, gated=True) == "64" and kind(4096, 8192, 4096, gated=True) == "256"
    assert kind(BIG, BIG, BIG) == "256"


def test_heights():
    for case, rows in (((8192, 4096, mq.MQ_BF16, False, False), 32), ((8192, 4096, mq.MQ_F32, False, False), 8),
                       ((8192, 4096, mq.MQ_F16, True, False), 8), ((4096, 4096, mq.MQ_BF16, False, False), 32), ((4095, 4032, mq.MQ_BF16, False, False), 8), ((500, 1000, mq.MQ_F16, False, False), 4),
                       ((300, 2700, mq.MQ_F16, False, True), 4), ((4096, 8192, mq.MQ_BF16, True, True), 8),
                       ((BIG, BIG, mq.MQ_BF16, False, False), 32)):
        assert quantize_height(*case) == rows, case
