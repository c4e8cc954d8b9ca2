"""The microscaled 4-bit calls refuse bad arguments on the host, before any launch (no GPU here); the
binding's constants match the header, the formulas of the gradients their differences, and the
validation runs clean under sanitizers (host code only, launchers stubbed)."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import microscaling_quantized_convolution_amd as mq
import mx4_reference as ref

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
S0 = ctypes.c_void_p(0)
OK, ARG, SHAPE = mq.MQ_OK, mq.MQ_ERR_ARG, mq.MQ_ERR_SHAPE
UNSUPPORTED, WORKSPACE = mq.MQ_ERR_UNSUPPORTED, mq.MQ_ERR_WORKSPACE
BIG = 1 << 30


def mat(rows, cols, dtype=mq.MQ_BF16, data=0x10000, stride=None):
    return mq.mq_matrix(data, cols if stride is None else stride, rows, cols, dtype)


def held(rows, cols, codes=0x20000, scales=0x30000):
    return mq.mq_mx4(rows, cols, codes, scales)


def test_header_constants_match_binding():
    hdr = open(os.path.join(ROOT, "include", "mq.h")).read()
    for name in ("MQ_F32", "MQ_MX4_BLOCK", "MQ_MX4_PIECE"):
        assert int(re.search(r"#define %s (\d+)" % name, hdr).group(1)) == getattr(mq, name)


def test_bytes():
    L = mq.lib()
    assert L.mq_mx4_codes_bytes(3, 256) == 3 * 128 and L.mq_mx4_codes_bytes(3, 257) == 2 * 3 * 128
    assert L.mq_mx4_scales_bytes(5, 1) == 40 and L.mq_mx4_scales_bytes(5, 513) == 120
    for bad in ((-1, 5), (5, -1), (0, 7), (7, 0)):
        assert L.mq_mx4_codes_bytes(*bad) == 0 and L.mq_mx4_scales_bytes(*bad) == 0
    assert L.mq_mx4_codes_bytes(BIG - 1, BIG - 1) == (BIG - 1) * (BIG // 256) * 128


WORKSPACES = ["matmul", "linear", "linear_backward", "gated", "gated_backward"]


@pytest.mark.parametrize("name", WORKSPACES)
def test_workspaces(name):
    f = getattr(mq.lib(), f"mq_mx4_{name}_workspace_bytes")
    sizes = [f(m, 300, 500) for m in range(0, 700, 7)]
    assert sizes == sorted(sizes)  # what suffices for m rows suffices for fewer
    for bad in ((-1, 4, 4), (4, -1, 4), (4, 4, -1), (BIG, 4, 4), (4, BIG, 4), (4, 4, BIG)):
        assert f(*bad) == 0


def test_quantize_refusals():
    def call(x=mat(4, 64), row=held(4, 64), col=held(64, 4), rnd=mq.MQ_RNE):
        return mq.lib().mq_mx4_quantize(x, row, col, rnd, 0, S0)
    for bad in (dict(x=None), dict(row=None, col=None), dict(rnd=2), dict(rnd=-1), dict(x=mat(4, 64, dtype=0)),
                dict(x=mat(4, 64, dtype=4)), dict(x=mat(-1, 64)), dict(x=mat(4, -64, stride=0)), dict(x=mat(4, 64, data=0)),
                dict(x=mat(4, 64, data=0x10001)), dict(x=mat(4, 64, mq.MQ_F32, 0x10002)), dict(x=mat(4, 64, stride=63)),
                dict(row=held(4, 64, codes=0)), dict(row=held(4, 64, scales=0)), dict(col=held(64, 4, codes=0x20008)),
                dict(col=held(64, 4, scales=0x30004)), dict(row=held(-4, 64))):
        assert call(**bad) == ARG, bad
    for bad in (dict(row=held(64, 4)), dict(col=held(4, 64)), dict(row=held(4, 63))):
        assert call(**bad) == SHAPE, bad
    assert call(x=mat(4, BIG), row=held(4, BIG), col=None) == UNSUPPORTED
    assert call(x=mat(0, 64, data=0), row=held(0, 64, 0, 0), col=held(64, 0, 0, 0)) == OK


def test_dequantize_refusals():
    f = lambda q=held(4, 64), out=mat(4, 64): mq.lib().mq_mx4_dequantize(q, out, S0)
    for bad in (dict(q=None), dict(out=None), dict(out=mat(4, 64, dtype=9)), dict(q=held(4, 64, codes=0x20001))):
        assert f(**bad) == ARG, bad
    assert f(out=mat(4, 65)) == SHAPE and f(q=held(0, 64, 0, 0), out=mat(0, 64, data=0)) == OK


def test_matmul_refusals():
    def call(a=held(4, 64), b=held(8, 64), y=mat(4, 8), ws=0x40000, size=1 << 40):
        return mq.lib().mq_mx4_matmul(a, b, y, ws, size, S0)
    for bad in (dict(a=None), dict(b=None), dict(y=None), dict(ws=0x40008), dict(y=mat(4, 8, stride=7))):
        assert call(**bad) == ARG, bad
    for bad in (dict(a=held(5, 64)), dict(b=held(8, 32)), dict(y=mat(4, 9))):
        assert call(**bad) == SHAPE, bad
    assert call(a=held(4, BIG), b=held(8, BIG)) == UNSUPPORTED
    assert call(a=held(0, 64, 0, 0), y=mat(0, 8, data=0)) == OK


def test_linear_refusals():
    need = mq.lib().mq_mx4_linear_workspace_bytes(4, 8, 64)
    assert need > 0

    def call(x=mat(4, 64), w=held(8, 64), y=mat(4, 8), x_col=None, ws=0x40000, size=need):
        return mq.lib().mq_mx4_linear(x, w, y, x_col, ws, size, S0)
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(x_col=held(64, 4, codes=0)), dict(ws=0x40001)):
        assert call(**bad) == ARG, bad
    for bad in (dict(x=mat(4, 63)), dict(y=mat(5, 8)), dict(y=mat(4, 9)), dict(x_col=held(4, 64))):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(ws=None), dict(size=need - 1)):
        assert call(**bad) == WORKSPACE, bad
    assert call(x=mat(4, BIG), w=held(8, BIG)) == UNSUPPORTED


def test_linear_backward_refusals():
    need = mq.lib().mq_mx4_linear_backward_workspace_bytes(4, 8, 64)

    def call(dy=mat(4, 8), x_col=held(64, 4), w_col=held(64, 8), dx=mat(4, 64), dw=mat(8, 64), rnd=1, ws=0x40000, size=need):
        return mq.lib().mq_mx4_linear_backward(dy, x_col, w_col, dx, dw, rnd, 3, ws, size, S0)
    for bad in (dict(dy=None), dict(dx=None, dw=None), dict(rnd=3), dict(x_col=None), dict(w_col=None), dict(ws=0x40004)):
        assert call(**bad) == ARG, bad
    for bad in (dict(dx=mat(4, 65)), dict(dw=mat(8, 65)), dict(dx=mat(5, 64)), dict(x_col=held(64, 5)),
                dict(w_col=held(64, 9)), dict(dw=mat(9, 64))):
        assert call(**bad) == SHAPE, bad
    assert call(ws=None) == WORKSPACE and call(size=need - 1) == WORKSPACE


def test_gated_refusals():
    need = mq.lib().mq_mx4_gated_workspace_bytes(4, 8, 64)

    def call(x=mat(4, 64), wg=held(8, 64), wu=held(8, 64), h=mat(4, 8), g=mat(4, 8), u=mat(4, 8), x_col=None,
             ws=0x40000, size=need):
        return mq.lib().mq_mx4_gated(x, wg, wu, h, g, u, x_col, ws, size, S0)
    for bad in (dict(x=None), dict(wg=None), dict(wu=None), dict(h=None), dict(g=None), dict(u=None), dict(ws=0x40002),
                dict(u=mat(4, 8, data=0))):
        assert call(**bad) == ARG, bad
    for bad in (dict(wg=held(9, 64)), dict(wu=held(8, 65)), dict(h=mat(5, 8)), dict(g=mat(4, 9)),
                dict(u=mat(4, 8, mq.MQ_F32)), dict(x_col=held(4, 64))):
        assert call(**bad) == SHAPE, bad
    assert call(ws=None) == WORKSPACE and call(size=need - 1) == WORKSPACE


def test_gated_backward_refusals():
    need = mq.lib().mq_mx4_gated_backward_workspace_bytes(4, 8, 64)

    def call(dh=mat(4, 8), g=mat(4, 8), u=mat(4, 8), x_col=held(64, 4), wg=held(64, 8), wu=held(64, 8), dx=mat(4, 64),
             dwg=mat(8, 64), dwu=mat(8, 64), rnd=0, ws=0x40000, size=need):
        return mq.lib().mq_mx4_gated_backward(dh, g, u, x_col, wg, wu, dx, dwg, dwu, rnd, 0, ws, size, S0)
    for bad in (dict(dh=None), dict(g=None), dict(u=None), dict(dwg=None), dict(dwu=None), dict(x_col=None), dict(wg=None),
                dict(wu=None), dict(rnd=5), dict(dx=None, dwg=None, dwu=None), dict(ws=0x40008)):
        assert call(**bad) == ARG, bad
    for bad in (dict(g=mat(4, 9)), dict(u=mat(4, 8, mq.MQ_F16)), dict(dx=mat(4, 63)), dict(wg=held(64, 9)),
                dict(dwu=mat(8, 65)), dict(dwu=mat(8, 64, mq.MQ_F32)), dict(x_col=held(64, 5))):
        assert call(**bad) == SHAPE, bad
    assert call(ws=None) == WORKSPACE and call(size=need - 1) == WORKSPACE


def test_gradient_formula_against_differences():
    """ref.gradients, which the kernels are held against, is the derivative of silu(g) u."""
    rng = np.random.default_rng(0)
    dh, g, u = rng.normal(size=(3, 500)) * np.array([[1], [4], [2]])
    dg, du = ref.gradients(dh, g, u)
    h = lambda a, b: a * ref.sigmoid(a) * b
    step = 1e-5
    # central differences: step^2 / 6 of a third derivative below 2 |u|, rounding 2^-53 / step of |h|
    near = 1e-9 * (1 + np.abs(dh)) * (1 + np.abs(g)) * (1 + np.abs(u))
    assert (np.abs(dg - dh * (h(g + step, u) - h(g - step, u)) / (2 * step)) <= near).all()
    assert (np.abs(du - dh * (h(g, u + step) - h(g, u - step)) / (2 * step)) <= near).all()


def test_reference_quantization():
    """The reference on blocks worked out by hand."""
    x = np.zeros((1, 64))
    x[0, :8] = [6, 5, 2.5, 0.25, 0.75, -3.5, -0.0, 1.25]
    x[0, 32:36] = [6.5, 1.5, -13, 0.1]
    code, e = ref.quantize(x)
    assert list(e[0, :2]) == [127, 129]  # 13 needs 4: 3.25
    assert list(code[0, :8]) == [7, 6, 4, 0, 2, 14, 8, 2]
    assert list(code[0, 32:36]) == [3, 1, 13, 0]  # 1.625 -> 1.5, .375 -> .5, 3.25 -> 3, .025 -> 0
    assert list(ref.rounded(x)[0, 32:36]) == [6, 2, -12, 0]
    # Philox4x32-10's published vectors: zeros, and all bits set
    ones = np.full((1, 4), 0xFFFFFFFF, dtype=np.uint64)
    assert [hex(v) for v in ref.philox(np.zeros((1, 4), dtype=np.uint64), (0, 0))[0]] == \
        ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    assert [hex(v) for v in ref.philox(ones, (0xFFFFFFFF, 0xFFFFFFFF))[0]] == \
        ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]


@pytest.mark.skipif(not os.path.isdir("/opt/rocm/include"), reason="needs the HIP headers")
def test_host_validation_under_sanitizers(tmp_path):
    exe = str(tmp_path / "mx4_asan")
    subprocess.check_call([
        "g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
        "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
        "-O1", "-g", os.path.join(HERE, "mx4_asan_driver.cpp"),
        os.path.join(ROOT, "microscaling_quantized_convolution_amd", "csrc", "mq_mx4_api.cpp"),
        "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "0 failures" in r.stdout and "runtime error" not in r.stderr
