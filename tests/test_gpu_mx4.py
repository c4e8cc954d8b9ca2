"""GPU tests of the microscaled 4-bit linear layers against their 64-bit definitions (mx4_reference):
quantization bit for bit, products exactly where fp32 sums are exact and within their bound
elsewhere, gradients within what a value next to a border of two codes may change."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_amd as mq
import mx4_reference as ref

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SHAPES = [(1, 1), (1, 32), (3, 31), (2, 33), (1, 4096), (33, 257), (257, 40), (256, 256), (70, 1000),
          (300, 513), (5, 8200), (1025, 96)]
# rows, columns and depth of products: one row to many, every size of tile cut on each side
PRODUCTS = [(1, 1, 1), (1, 64, 256), (1, 4096, 4096), (2, 17, 300), (7, 100, 32), (16, 512, 2048),
            (17, 129, 257), (33, 70, 8192), (40, 1111, 2000), (65, 64, 64), (100, 300, 511), (129, 500, 1024),
            (300, 257, 768), (128, 128, 4096), (512, 512, 512), (513, 1030, 300), (1500, 1025, 260), (37, 2050, 33)]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def dense(seed, rows, cols, dtype=F32, spread=0.0):
    g = gen(seed)
    x = torch.randn(rows, cols, generator=g)
    return (x * torch.exp(spread * torch.randn(rows, 1, generator=g))).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def held(code, e, cols):
    """A quantized matrix on the GPU from the reference's codes."""
    codes, scales = ref.packed(code, e)
    return mq.MX4(code.shape[0], cols, codes.cuda(), scales.cuda())


def same(q, code, e):
    codes, scales = ref.packed(code, e)
    assert torch.equal(q.scales.cpu(), scales), "scales"
    assert torch.equal(q.codes.cpu(), codes), "codes"


def random_codes(seed, rows, cols, low=126, high=128):
    """Codes of every kind, scales of [low, high], the columns past the last zero."""
    rng = np.random.default_rng(seed)
    width = -(-cols // 256) * 256
    code = rng.integers(0, 16, (rows, width))
    code[:, cols:] = 0
    return code, rng.integers(low, high + 1, (rows, width // 32))


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(rows, cols, dtype):
    x = dense(rows * 7 + cols, rows, cols, dtype, 1.0)
    row, col = mq.MX4.empty(rows, cols), mq.MX4.empty(cols, rows)
    for q in (row, col):
        q.codes.fill_(0x77), q.scales.fill_(0x77)
    mq.mq_mx4_quantize(x.cuda(), row, col)
    same(row, *ref.quantize(f64(x)))
    same(col, *ref.quantize(f64(x).T))
    # one direction alone: the same bytes
    for r, c in ((True, False), (False, True)):
        one = mq.MX4.empty(rows, cols) if r else mq.MX4.empty(cols, rows)
        mq.mq_mx4_quantize(x.cuda(), one if r else None, one if c else None)
        other = row if r else col
        assert torch.equal(one.codes, other.codes) and torch.equal(one.scales, other.scales)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 50), (65, 129), (300, 513), (256, 512)])
def test_quantize_stochastic(rows, cols, dtype):
    x, seed = dense(rows + cols, rows, cols, dtype, 1.0), 0x123456789ABCDEF
    row, col = mq.MX4.empty(rows, cols), mq.MX4.empty(cols, rows)
    mq.mq_mx4_quantize(x.cuda(), row, col, mq.MQ_SR, seed)
    same(row, *ref.quantize(f64(x), seed, 0))
    same(col, *ref.quantize(f64(x).T, seed, 1))


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
def test_quantize_every_sixteen_bit_value(dtype):
    """Every bf16 or f16 bit pattern (for fp32: every upper half, with all kinds of lower halves) as
    an element, in blocks of like magnitude, NaN and infinities among them; and every border."""
    bits = torch.arange(65536, dtype=torch.int32)
    if dtype == F32:
        low = torch.randint(0, 65536, (65536,), generator=gen(1), dtype=torch.int32)
        x = ((bits << 16) | low).view(F32)
    else:
        x = bits.to(torch.uint16).view(dtype)
    x = x.reshape(-1, 32)
    x = torch.cat([x, torch.flip(x[:, :16], [1]).repeat(1, 2)])
    edges = torch.tensor([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, -.25, -.75, -1.25, -1.75, -2.5,
                          -3.5, -5, -6, -0.0, 5.96875, 3.015625, 0.2490234375, 0.2509765625, 4.96875, 5.03125, 2.484375, 1])
    x = torch.cat([x, (edges * torch.tensor([1.0, 2.0 ** -10, 2.0 ** 9, 2.0 ** -14])[:, None]).to(dtype)])
    row, col = mq.MX4.empty(*x.shape), mq.MX4.empty(x.shape[1], x.shape[0])
    mq.mq_mx4_quantize(x.cuda(), row, col)
    same(row, *ref.quantize(f64(x)))
    same(col, *ref.quantize(f64(x).T))


def test_quantize_extremes():
    """Zeros, the smallest and largest numbers, NaN and infinities in single blocks."""
    top = torch.finfo(F32).max
    x = torch.zeros(9, 96)
    x[1, 0], x[1, 40], x[2, 5] = -0.0, 1e-45, 2.0 ** -126
    x[3, 7], x[3, 8], x[3, 50] = top, -top / 3, top
    x[4, 1], x[4, 33] = float("nan"), 1.0
    x[5, 64], x[5, 0] = float("inf"), 3.0
    x[6, 95], x[6, 1] = -float("inf"), -3.0
    x[7] = 6.0 * 2.0 ** -125
    x[8] = -7.0
    for sr in (None, 99):
        row, col = mq.MX4.empty(9, 96), mq.MX4.empty(96, 9)
        mq.mq_mx4_quantize(x.cuda(), row, col, mq.MQ_RNE if sr is None else mq.MQ_SR, sr or 0)
        same(row, *ref.quantize(f64(x), sr, 0))
        same(col, *ref.quantize(f64(x).T, sr, 1))
        for dtype in (F32, BF16):
            out = mq.mq_mx4_dequantize(row, torch.empty(9, 96, dtype=dtype, device="cuda"))
            want = torch.from_numpy(ref.rounded(f64(x), sr, 0)).to(dtype)
            assert torch.equal(out.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
def test_views(dtype):
    """Rows of every alignment inside a larger matrix; what lies around outputs stays."""
    big = dense(5, 90, 700, dtype).cuda()
    for r0, c0, rows, cols in ((1, 1, 40, 300), (0, 8, 64, 256), (3, 2, 33, 77), (2, 16, 80, 601)):
        x = big[r0:r0 + rows, c0:c0 + cols]
        row, col = mq.MX4.empty(rows, cols), mq.MX4.empty(cols, rows)
        mq.mq_mx4_quantize(x, row, col)
        same(row, *ref.quantize(f64(x)))
        same(col, *ref.quantize(f64(x).T))
        out = torch.full((100, 720), 3.0, dtype=dtype, device="cuda")
        view = out[r0 + 1:r0 + 1 + rows, c0 + 1:c0 + 1 + cols]
        mq.mq_mx4_dequantize(row, view)
        assert torch.equal(view.cpu(), torch.from_numpy(ref.rounded(f64(x))).to(dtype))
        view.fill_(3.0)
        assert (out == 3.0).all()
        w = random_codes(r0, 50, cols)
        y = torch.full((100, 70), 3.0, dtype=dtype, device="cuda")
        at = y[r0 + 1:r0 + 1 + rows, c0 + 1:c0 + 51]
        mq.mq_mx4_linear(x, held(*w, cols), at, mq.mx4_linear_workspace(rows, 50, cols))
        want, bound = ref.product(ref.rounded(f64(x)), ref.values(*w, cols))
        assert (np.abs(f64(at) - want) <= bound + ref.half_step(dtype, np.abs(want) + bound)).all()
        at.fill_(3.0)
        assert (y == 3.0).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_matmul(m, n, k, dtype):
    """Terms are multiples of 2^-4 and their sums stay below 2^20, so that every fp32 sum is exact."""
    a, b = random_codes(m + n, m, k), random_codes(m * n + k, n, k)
    y = torch.full((m, n), float("nan"), dtype=dtype, device="cuda")
    mq.mq_mx4_matmul(held(*a, k), held(*b, k), y, mq.mx4_matmul_workspace(m, n, k))
    va, vb = ref.values(*a, k), ref.values(*b, k)
    want = va @ vb.T
    assert np.abs(va).max() * np.abs(vb).max() <= 144 and (np.abs(va) @ np.abs(vb).T).max() < 2.0 ** 20
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(F32).to(dtype))


@pytest.mark.parametrize("m,n,k", [(5, 300, 4096), (130, 130, 8192), (600, 300, 2048)])
def test_matmul_wide_scales(m, n, k):
    a, b = random_codes(1, m, k, 100, 150), random_codes(2, n, k, 90, 160)
    y = torch.empty(m, n, device="cuda")
    mq.mq_mx4_matmul(held(*a, k), held(*b, k), y, mq.mx4_matmul_workspace(m, n, k))
    want, bound = ref.product(ref.values(*a, k), ref.values(*b, k))
    assert (np.abs(f64(y) - want) <= bound).all()


@pytest.mark.parametrize("m,n,k", [(3, 40, 300), (50, 300, 1000), (300, 300, 1024)])
def test_nan_blocks(m, n, k):
    """A block with scale 255 makes the sums that it takes part in NaN, and no others."""
    a, b = random_codes(3, m, k), random_codes(4, n, k)
    a[1][1, 0], b[1][7, (k - 1) // 32], b[1][n - 1, 0] = 255, 255, 255
    a[0][1, :32], b[0][n - 1, :32] = 0, 0
    y = torch.empty(m, n, device="cuda")
    mq.mq_mx4_matmul(held(*a, k), held(*b, k), y, mq.mx4_matmul_workspace(m, n, k))
    want = torch.from_numpy(ref.values(*a, k) @ ref.values(*b, k).T).to(F32)
    assert torch.isnan(y.cpu()).eq(torch.isnan(want)).all()
    assert torch.equal(y.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("x_dtype,y_dtype", [(BF16, BF16), (F16, F32), (F32, F16), (BF16, F32)])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_linear(m, n, k, x_dtype, y_dtype):
    x, w = dense(m + k, m, k, x_dtype, 0.5), random_codes(n, n, k)
    y = torch.full((m, n), float("nan"), dtype=y_dtype, device="cuda")
    x_col = mq.MX4.empty(k, m)
    mq.mq_mx4_linear(x.cuda(), held(*w, k), y, mq.mx4_linear_workspace(m, n, k), x_col)
    want, bound = ref.product(ref.rounded(f64(x)), ref.values(*w, k))
    assert (np.abs(f64(y) - want) <= bound + ref.half_step(y_dtype, np.abs(want) + bound)).all()
    same(x_col, *ref.quantize(f64(x).T))
    # without the columns, and as two calls: the same bits
    z, row = torch.empty_like(y), mq.MX4.empty(m, k)
    mq.mq_mx4_linear(x.cuda(), held(*w, k), z, mq.mx4_linear_workspace(m, n, k))
    assert torch.equal(y, z)
    mq.mq_mx4_quantize(x.cuda(), row)
    mq.mq_mx4_matmul(row, held(*w, k), z, mq.mx4_matmul_workspace(m, n, k))
    assert torch.equal(y, z)


@pytest.mark.parametrize("dtype,w_dtype", [(BF16, F32), (F16, F16), (F32, BF16)])
@pytest.mark.parametrize("sr", [None, 77], ids=["nearest", "stochastic"])
@pytest.mark.parametrize("m,n,k", [(1, 33, 40), (8, 512, 256), (100, 300, 70), (257, 256, 512), (1000, 130, 300)])
def test_linear_backward(m, n, k, sr, dtype, w_dtype):
    dy, x, w = dense(m, m, n, dtype, 1.0), dense(n, m, k), dense(k, n, k)
    x_col, w_col = ref.quantize(f64(x).T), ref.quantize(f64(w).T)
    dx = torch.full((m, k), float("nan"), dtype=dtype, device="cuda")
    dw = torch.full((n, k), float("nan"), dtype=w_dtype, device="cuda")
    rnd, seed = (mq.MQ_RNE, 0) if sr is None else (mq.MQ_SR, sr)
    xq, wq, ws = held(*x_col, m), held(*w_col, n), mq.mx4_linear_backward_workspace(m, n, k)
    mq.mq_mx4_linear_backward(dy.cuda(), xq, wq, dx, dw, ws, rnd, seed)
    for got, a, b in ((dx, ref.rounded(f64(dy), sr, 0), ref.values(*w_col, n)),
                      (dw, ref.rounded(f64(dy).T, sr, 1), ref.values(*x_col, m))):
        want, bound = ref.product(a, b)
        assert (np.abs(f64(got) - want) <= bound + ref.half_step(got.dtype, np.abs(want) + bound)).all()
    # either one alone: the same bits
    one = torch.empty_like(dx)
    mq.mq_mx4_linear_backward(dy.cuda(), None, wq, one, None, ws, rnd, seed)
    assert torch.equal(one, dx)
    one = torch.empty_like(dw)
    mq.mq_mx4_linear_backward(dy.cuda(), xq, None, None, one, ws, rnd, seed)
    assert torch.equal(one, dw)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,f,k", [(1, 1, 1), (1, 300, 512), (4, 1030, 2048), (16, 256, 256), (17, 65, 100), (33, 200, 700),
                                   (100, 129, 300), (257, 300, 512), (600, 520, 260)])
def test_gated(m, f, k, dtype):
    x, wg, wu = dense(m, m, k, dtype, 0.3), dense(f, f, k) / k ** 0.5 * 2, dense(k, f, k) / k ** 0.5
    wg, wu = ref.quantize(f64(wg)), ref.quantize(f64(wu))
    ws = mq.mx4_gated_workspace(m, f, k)
    h, g, u = (torch.full((m, f), float("nan"), dtype=dtype, device="cuda") for _ in range(3))
    x_col = mq.MX4.empty(k, m)
    mq.mq_mx4_gated(x.cuda(), held(*wg, k), held(*wu, k), h, ws, g, u, x_col)
    same(x_col, *ref.quantize(f64(x).T))
    xq = ref.rounded(f64(x))
    (rg, bg), (ru, bu) = ref.product(xq, ref.values(*wg, k)), ref.product(xq, ref.values(*wu, k))
    for got, want, bound in ((g, rg, bg), (u, ru, bu)):
        assert (np.abs(f64(got) - want) <= bound + ref.half_step(dtype, np.abs(want) + bound)).all()
    s = ref.sigmoid(rg)
    want = rg * s * ru
    # |silu'| < 1.1; the activation's own fp32 operations: 16 of 2^-23, the exponential's argument
    # |g| 2^-22 times the slope |g (1 - s)| of silu's logarithm
    bound = 1.1 * bg * (np.abs(ru) + bu) + np.abs(rg * s) * bu + np.abs(want) * (16 * 2.0 ** -23 + np.abs(rg) * 2.0 ** -22)
    assert (np.abs(f64(h) - want) <= bound + ref.half_step(dtype, np.abs(want) + bound)).all()
    alone = torch.empty_like(h)
    mq.mq_mx4_gated(x.cuda(), held(*wg, k), held(*wu, k), alone, ws)
    assert torch.equal(alone, h)


def test_gated_far_values():
    """Gates far below and above zero, infinite and NaN ones."""
    big = 2.0 ** 60
    x = torch.zeros(6, 32)
    x[:, 0] = torch.tensor([1.0, -1.0, 30.0, -30.0, 120.0, float("nan")])
    wg, wu = torch.zeros(3, 32), torch.zeros(3, 32)
    wg[:, 0], wu[:, 0] = torch.tensor([1.0, 4.0, big]), torch.tensor([1.0, 2.0, 1.0])
    qs = [mq.MX4.empty(3, 32) for _ in range(2)]
    for w, q in zip((wg, wu), qs):
        mq.mq_mx4_quantize(w.cuda(), q)
    h = torch.empty(6, 3, device="cuda")
    mq.mq_mx4_gated(x.cuda(), *qs, h, mq.mx4_gated_workspace(6, 3, 32))
    xq = ref.rounded(f64(x))
    g, u = xq @ f64(wg).T, xq @ f64(wu).T
    want = g * ref.sigmoid(g) * u
    h = f64(h)
    assert np.isnan(h[5]).all() and np.isfinite(h[:5]).all()
    tiny = 2.0 ** -100  # what exponentials below the range of fp32 leave
    assert (np.abs(h[:5] - want[:5]) <= np.abs(want[:5]) * (16 + np.abs(np.clip(g[:5], -90, 90))) * 2.0 ** -22 + tiny).all()


@pytest.mark.parametrize("dtype,w_dtype", [(BF16, BF16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("m,f,k", [(1, 33, 40), (8, 512, 256), (100, 300, 70), (257, 256, 300), (700, 130, 257)])
def test_gated_backward(m, f, k, dtype, w_dtype):
    dh, g, u = dense(m, m, f, dtype, 0.5), (2 * dense(f, m, f)).to(dtype), dense(k, m, f, dtype)
    x, wg, wu = dense(4, m, k), dense(5, f, k), dense(6, f, k)
    x_col, wg_col, wu_col = (ref.quantize(f64(t).T) for t in (x, wg, wu))
    dx = torch.full((m, k), float("nan"), dtype=dtype, device="cuda")
    dwg, dwu = (torch.full((f, k), float("nan"), dtype=w_dtype, device="cuda") for _ in range(2))
    ws = mq.mx4_gated_backward_workspace(m, f, k)
    args = [dh.cuda(), g.cuda(), u.cuda()]
    hq = held(*x_col, m), held(*wg_col, f), held(*wu_col, f)
    mq.mq_mx4_gated_backward(*args, *hq, dx, dwg, dwu, ws)
    dg, du = ref.gradients(f64(dh), f64(g), f64(u))
    s = ref.sigmoid(f64(g))
    off_g, off_u = np.abs(f64(dh) * f64(u)) * ref.LOOSE, np.abs(f64(dh) * f64(g) * s) * ref.LOOSE

    def part(v, off, w):
        want, bound = ref.product(ref.rounded(v), w)
        return want, bound + ref.unsure(v, off) @ np.abs(w).T
    xv = ref.values(*x_col, m)
    parts = [part(dg, off_g, ref.values(*wg_col, f)), part(du, off_u, ref.values(*wu_col, f))]
    for got, want, bound in ((dx, parts[0][0] + parts[1][0], (parts[0][1] + parts[1][1]) * 2),
                             (dwg, *part(dg.T, off_g.T, xv)), (dwu, *part(du.T, off_u.T, xv))):
        bound = bound + ref.half_step(got.dtype, np.abs(want) + bound)
        assert (np.abs(f64(got) - want) <= bound).all()
    # either side alone: the same bits
    one = torch.empty_like(dx)
    mq.mq_mx4_gated_backward(*args, None, *hq[1:], one, None, None, ws)
    assert torch.equal(one, dx)
    two = torch.empty_like(dwg), torch.empty_like(dwu)
    mq.mq_mx4_gated_backward(*args, hq[0], None, None, None, *two, ws)
    assert torch.equal(two[0], dwg) and torch.equal(two[1], dwu)


def test_gated_backward_stochastic():
    """With u = 0 (so dg = 0) and g large and negative or positive (s = 0 or 1 exactly), du is dh * g or
    0, both exact: what is left is the rounding, by the draws of direction 2 and 3."""
    m, f, k, seed = 70, 300, 130, 1 << 40 | 5
    dh, g = dense(1, m, f, BF16), torch.full((m, f), 128.0, dtype=BF16)
    g[::3] = -256.0
    u = torch.zeros(m, f, dtype=BF16)
    x, w = dense(4, m, k), dense(5, f, k)
    x_col, w_col = ref.quantize(f64(x).T), ref.quantize(f64(w).T)
    dx, dwg, dwu = (torch.empty(*s, device="cuda") for s in ((m, k), (f, k), (f, k)))
    mq.mq_mx4_gated_backward(dh.cuda(), g.cuda(), u.cuda(), held(*x_col, m), held(*w_col, f), held(*w_col, f),
                             dx, dwg, dwu, mq.mx4_gated_backward_workspace(m, f, k), mq.MQ_SR, seed)
    du = f64(dh) * np.where(f64(g) > 0, f64(g), 0.0)
    for got, a, b in ((dx, ref.rounded(du, seed, 2), ref.values(*w_col, f)),
                      (dwu, ref.rounded(du.T, seed, 3), ref.values(*x_col, m))):
        want, bound = ref.product(a, b)
        assert (np.abs(f64(got) - want) <= bound).all()
    assert (dwg == 0).all()


def test_empty():
    """No rows, no outputs, and sums of nothing."""
    z = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")
    w = held(*random_codes(1, 20, 64), 64)
    mq.mq_mx4_linear(z(0, 64), w, z(0, 20), mq.mx4_linear_workspace(0, 20, 64), mq.MX4.empty(64, 0))
    mq.mq_mx4_quantize(z(0, 64), mq.MX4.empty(0, 64), mq.MX4.empty(64, 0))
    mq.mq_mx4_quantize(z(3, 0), mq.MX4.empty(3, 0), mq.MX4.empty(0, 3))
    assert mq.mq_mx4_dequantize(mq.MX4.empty(0, 5), z(0, 5)).shape == (0, 5)
    for m, n in ((3, 20), (300, 400), (1, 1)):
        y = torch.full((m, n), float("nan"), device="cuda")
        mq.mq_mx4_matmul(mq.MX4.empty(m, 0), mq.MX4.empty(n, 0), y, mq.mx4_matmul_workspace(m, n, 0))
        assert (y == 0).all()
    dw, dx = torch.full((20, 64), 7.0, device="cuda"), z(0, 64)
    ws = mq.mx4_linear_backward_workspace(0, 20, 64)
    w_col = held(*random_codes(1, 64, 20), 20)
    mq.mq_mx4_linear_backward(z(0, 20), mq.MX4.empty(64, 0), w_col, dx, dw, ws)
    assert (dw == 0).all()
    dwg, dwu = (torch.full((20, 64), 7.0, device="cuda") for _ in range(2))
    mq.mq_mx4_gated_backward(z(0, 20), z(0, 20), z(0, 20), mq.MX4.empty(64, 0), w_col, w_col, dx, dwg, dwu,
                             mq.mx4_gated_backward_workspace(0, 20, 64))
    assert (dwg == 0).all() and (dwu == 0).all()
    mq.mq_mx4_gated(z(0, 64), w, w, z(0, 20), mq.mx4_gated_workspace(0, 20, 64))


def test_larger_workspace_serves_fewer_rows():
    n, k = 300, 512
    w = random_codes(1, n, k)
    ws = mq.mx4_linear_workspace(700, n, k)
    for m in (700, 513, 256, 129, 64, 33, 16, 3, 1):
        x, y = dense(m, m, k, BF16), torch.empty(m, n, device="cuda")
        mq.mq_mx4_linear(x.cuda(), held(*w, k), y, ws)
        want, bound = ref.product(ref.rounded(f64(x)), ref.values(*w, k))
        assert (np.abs(f64(y) - want) <= bound).all(), m
