"""GPU tests of the 4-bit products in every kernel that their rule takes, and of the quantization in every
height of its register tiles: whole results, in every type, with edges that no tile divides. The rule itself
says which kernel a size takes, so that sizes cannot be left behind by it."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_amd as mq
import mx4_reference as ref
from test_gpu_mx4 import BF16, F16, F32, f64, same
from test_gpu_mx4_reach import check_rows, random_held, some
from test_mx4_limits import KINDS, matmul_kind, quantize_height

pytestmark = pytest.mark.gpu
TYPES = [BF16, F16, F32]
MQ_TYPE = {BF16: mq.MQ_BF16, F16: mq.MQ_F16, F32: mq.MQ_F32}
ids = {BF16: "bf16", F16: "f16", F32: "f32"}.get
by_type = pytest.mark.parametrize("dtype", TYPES, ids=ids)


def values(q):
    """A quantized matrix on the GPU in 64 bits."""
    grid = torch.tensor(np.concatenate([ref.GRID, -ref.GRID]), device="cuda")
    codes = torch.stack([q.codes & 15, q.codes >> 4], 3).long()  # [pieces][rows][128][2]
    pieces, rows = codes.shape[:2]
    v = grid[codes].view(pieces, rows, 8, 32) * torch.exp2(q.scales.double() - 127)[..., None]
    return v.permute(1, 0, 2, 3).reshape(rows, pieces * 256)[:, :q.shape[1]]


def product(*pairs):
    """sum of a b^T in 64 bits. Also asserts that every sum in fp32 is exact: all terms are multiples of one
    unit, and the magnitudes together stay below 2^24 of it."""
    total = sum(torch.mm(a, b.t().contiguous()) for a, b in pairs)
    unit = min(step(a) * step(b) for a, b in pairs)
    assert sum(torch.mm(a.abs(), b.abs().t().contiguous()).max().item() for a, b in pairs) < 2 ** 24 * unit
    return total


def step(v):
    """The largest power of two, up to 1024, that all of v are multiples of."""
    unit = 1024.0
    while not torch.equal(torch.round(v / unit), v / unit):
        unit /= 2
    return unit


def grid(seed, rows, cols, dtype, factor=1.0):
    """A dense matrix of the elements' own values, which every block of rows and of columns holds exactly: a
    smaller scale's elements have all those of a larger one that it reaches."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    v = torch.cat([v, -v])
    return (v[torch.randint(0, 16, (rows, cols), generator=g, device="cuda")] * factor).to(dtype)


def inside(rows, cols, dtype, lines=False):
    """Room for an output in the midst of a larger matrix, at no alignment but the elements' own, or with
    rows that begin with a line of memory."""
    around, at = (-cols % 128 + 256, 128) if lines else (7, 3)
    big = torch.full((rows + 3, cols + around), 3.0, dtype=dtype, device="cuda")
    return big, big[1:1 + rows, at:at + cols]


def check(out, want):
    big, view = out
    assert torch.equal(view, want.to(F32).to(view.dtype))
    view.fill_(3.0)
    assert (big == 3.0).all()


def kind(m, n, k, jobs=1, gated=False, sums=1):
    return KINDS[matmul_kind(jobs, m, n, sums * -(-k // 256), gated)]


# one size to each kernel, twice the largest: outputs of 86 MB and more pass the caches where rows begin with a
# line of memory, those of 172 MB anyhow
by_lines = pytest.mark.parametrize("lines", [False, True], ids=["any", "lines"])
PRODUCTS = [("rows", 13, 5001, 700), ("64", 333, 1111, 2001), ("128 deep", 1500, 1900, 700), ("128", 2300, 2900, 300),
            ("256", 4001, 3999, 1001), ("256", 6501, 6603, 1500)]


@by_type
@by_lines
@pytest.mark.parametrize("name,m,n,k", PRODUCTS)
def test_matmul(name, m, n, k, lines, dtype):
    assert kind(m, n, k) == name
    a, b, out = random_held(m, m, k), random_held(n + 1, n, k), inside(m, n, dtype, lines)
    mq.mq_mx4_matmul(a, b, out[1])
    check(out, product((values(a), values(b))))


@pytest.mark.parametrize("name,m,n,k", PRODUCTS[:5])
def test_matmul_nan(name, m, n, k):
    """Blocks of scale 255 in the first, a middle and the last rows, columns and blocks."""
    a, b, y = random_held(m, m, k), random_held(n + 1, n, k), torch.empty(m, n, dtype=BF16, device="cuda")
    rows, cols = [0, m // 2 + 1, m - 1], [0, n // 3, n - 1]
    last = (k - 1) // 32
    for q, at in ((a, rows), (b, cols)):
        for r, block in zip(at, (last, 3, 0)):
            q.scales[block // 8, r, block % 8] = 255
            q.codes[block // 8, r, block % 8 * 16:block % 8 * 16 + 16] = 0
    mq.mq_mx4_matmul(a, b, y)
    for q in (a, b):
        q.scales[q.scales == 255] = 127  # (of codes that are 0)
    want = product((values(a), values(b)))
    want[rows], want[:, cols] = float("nan"), float("nan")
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(y.nan_to_num(7.0), want.to(F32).to(BF16).nan_to_num(7.0))


GATED = [("rows", 5, 3001, 700, True), ("64", 300, 2001, 700, True), ("128 deep", 1000, 1500, 700, True),
         ("128", 2300, 1600, 300, True), ("256", 4001, 1999, 1001, True), ("256", 4001, 1999, 1001, False),
         ("256", 5001, 2999, 1300, True)]


@by_type
@by_lines
@pytest.mark.parametrize("name,m,f,k,keep", GATED)
def test_gated(name, m, f, k, keep, lines, dtype):
    assert kind(m, f, k, gated=True) == name
    x, wg, wu = grid(m, m, k, dtype), random_held(2, f, k), random_held(3, f, k)
    wg.scales -= 6
    wu.scales -= 4
    h, g, u = (inside(m, f, dtype, lines) for _ in range(3))
    ws = mq.mx4_gated_workspace(m, f, k)
    mq.mq_mx4_gated(x, wg, wu, h[1], ws, *((g[1], u[1]) if keep else ()))
    rg, ru = product((x.double(), values(wg))), product((x.double(), values(wu)))
    want = rg / (1 + torch.exp(-rg)) * ru
    # the sums are exact; the activation's own fp32 operations: 16 of 2^-23, and the exponential's argument, off
    # by |g| 2^-22 at most; h is rounded once
    info = torch.finfo(dtype)
    off = want.abs() * (16 * 2.0 ** -23 + rg.abs().clamp(max=200) * 2.0 ** -22) + ru.abs() * 2.0 ** -100 + 2.0 ** -126
    half = torch.clamp((want.abs() + off) * (info.eps / 2), min=info.smallest_normal * info.eps / 2)
    assert want.abs().max() < info.max / 2
    assert ((h[1].double() - want).abs() <= off + half).all()
    h[1].fill_(3.0)
    assert (h[0] == 3.0).all()
    if keep:
        check(g, rg)
        check(u, ru)
        alone = torch.empty(m, f, dtype=dtype, device="cuda")
        again = torch.empty(m, f, dtype=dtype, device="cuda")
        mq.mq_mx4_gated(x, wg, wu, alone, ws)
        mq.mq_mx4_gated(x, wg, wu, again, ws, torch.empty_like(again), torch.empty_like(again))
        assert torch.equal(alone, again)


@pytest.mark.parametrize("dtype,w_dtype", [(BF16, F16), (F16, F32), (F32, BF16)], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("names,m,n,k", [(("256", "128 deep"), 4001, 1001, 3999), (("128 deep", "256"), 1001, 4001, 3999),
                                         (("128", "64"), 3001, 300, 2301), (("rows", "rows"), 9, 13, 3001),
                                         (("128 deep", "rows"), 600, 13, 5001)])
def test_linear_backward(names, m, n, k, dtype, w_dtype):
    assert (kind(m, k, n), kind(n, k, m)) == names
    dy, x_col, w_col = grid(1, m, n, dtype, 0.25), random_held(2, k, m), random_held(3, k, n)
    dx, dw = inside(m, k, dtype), inside(n, k, w_dtype)
    mq.mq_mx4_linear_backward(dy, x_col, w_col, dx[1], dw[1], mq.mx4_linear_backward_workspace(m, n, k))
    d = dy.double()
    check(dx, product((d, values(w_col))))
    check(dw, product((d.t(), values(x_col))))


@pytest.mark.parametrize("dtype,w_dtype", [(BF16, BF16), (F16, F32), (F32, F16)], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("names,m,f,k", [(("256", "128 deep"), 4001, 500, 3999), (("128 deep", "256"), 1001, 4001, 3999),
                                         (("128", "64"), 3001, 300, 2301), (("rows", "64"), 9, 300, 3001),
                                         (("128 deep", "rows"), 600, 13, 4001)])
@by_lines
def test_gated_backward(names, m, f, k, lines, dtype, w_dtype):
    """With g of 32 (s = 1, 1 - s = 0 in fp32) or -256 (s = 0) and u of +-2, dg and du are dh times a power of
    two, or 0: exact, and what is quantized is exact too."""
    assert (kind(m, k, f, sums=2), kind(f, k, m, jobs=2)) == names
    dh, u = grid(1, m, f, dtype, 0.25), torch.full((m, f), 2.0, dtype=dtype, device="cuda")
    g = torch.full((m, f), 32.0, dtype=dtype, device="cuda")
    g[::3, ::2] = -256.0
    u[:, 1::3] = -2.0
    x_col, wg_col, wu_col = random_held(2, k, m), random_held(3, k, f), random_held(4, k, f)
    wu_col.scales -= 4  # du is 16 times dg
    dx, dwg, dwu = inside(m, k, dtype, lines), inside(f, k, w_dtype, lines), inside(f, k, w_dtype, lines)
    mq.mq_mx4_gated_backward(dh, g, u, x_col, wg_col, wu_col, dx[1], dwg[1], dwu[1],
                             mq.mx4_gated_backward_workspace(m, f, k))
    on = (g > 0).double()
    dg, du = dh.double() * u.double() * on, dh.double() * 32.0 * on
    check(dx, product((dg, values(wg_col)), (du, values(wu_col))))
    check(dwg, product((dg.t(), values(x_col))))
    check(dwu, product((du.t(), values(x_col))))


# ---- quantization --------------------------------------------------------------------------------

HEIGHTS = [(70, 131105), (33, 131072), (130, 22001), (300, 513)]


def spread(seed, rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") *
            torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))).to(dtype)


@pytest.mark.parametrize("sr", [None, 31 << 40 | 7], ids=["nearest", "stochastic"])
@by_type
@pytest.mark.parametrize("rows,cols", HEIGHTS)
def test_quantize(rows, cols, dtype, sr):
    """Both directions, every byte, at each height of the tiles."""
    tall = 32 if sr is None and dtype != F32 else 8
    assert quantize_height(rows, cols, MQ_TYPE[dtype], sr is not None, False) == \
        {131105: tall, 131072: tall, 22001: 8, 513: 4}[cols]
    x = spread(rows, rows, cols, dtype)
    row, col = mq.MX4.empty(rows, cols), mq.MX4.empty(cols, rows)
    for q in (row, col):
        q.codes.fill_(0x77), q.scales.fill_(0x77)
    rounding = (mq.MQ_RNE, 0) if sr is None else (mq.MQ_SR, sr)
    mq.mq_mx4_quantize(x, row, col, *rounding)
    same(row, *ref.quantize(f64(x), sr, 0))
    same(col, *ref.quantize(f64(x).T, sr, 1))
    alone = mq.MX4.empty(cols, rows)
    mq.mq_mx4_quantize(x, None, alone, *rounding)
    assert torch.equal(alone.codes, col.codes) and torch.equal(alone.scales, col.scales)


@pytest.mark.parametrize("rows,cols,dtype,sr", [(4200, 4096, F32, None), (4200, 4096, F32, 77), (8200, 4104, BF16, 77),
                                                (16500, 2056, F16, 1 << 50)])
def test_quantize_large_inputs(rows, cols, dtype, sr):
    """Inputs of 64 MiB whose rows begin with a line of memory, which are read past the caches: the bytes of the
    same input at another place, which is not, and of some rows' and columns' definition."""
    assert quantize_height(rows, cols, MQ_TYPE[dtype], sr is not None, False) == 8
    wide = -cols % 32 + 32 + cols
    place = torch.zeros(rows, wide, dtype=dtype, device="cuda")
    x, other = place[:, :cols], torch.zeros(rows, wide + 1, dtype=dtype, device="cuda")[:, 1:cols + 1]
    x.copy_(spread(1, rows, cols, dtype))
    x[5, 100], x[rows - 1, cols - 1] = float("inf"), float("nan")
    other.copy_(x)
    assert x.data_ptr() % 64 == 0 and x.stride(0) * x.element_size() % 64 == 0 and x.numel() * x.element_size() >= 64 << 20
    rounding = (mq.MQ_RNE, 0) if sr is None else (mq.MQ_SR, sr)
    held = []
    for t in (x, other):
        row, col = mq.MX4.empty(rows, cols), mq.MX4.empty(cols, rows)
        mq.mq_mx4_quantize(t, row, col, *rounding)
        held.append((row, col))
    for a, b in zip(*held):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    if sr is None:
        at = some(rows)
        check_rows(held[0][0], at, *ref.quantize(f64(x[at])))
        at = some(cols)
        check_rows(held[0][1], at, *ref.quantize(f64(x[:, at]).T))


def special(rows, cols, dtype):
    """Every bit pattern of 16 bits (fp32: every upper half), like ones in one block of a row and of a column;
    below them values at the borders of codes, NaN, infinities, zeros and the smallest numbers."""
    lane = torch.arange(32)[:, None] + torch.arange(65536)
    bits = (torch.arange(65536) & ~31) | (lane & 31)  # [32][65536]: a block's patterns, in another order to each row
    if dtype == F32:
        low = torch.randint(0, 65536, bits.shape, generator=torch.Generator().manual_seed(1))
        top = (((bits << 16) | low) & 0xFFFFFFFF)
        top = torch.where(top >= 1 << 31, top - (1 << 32), top).to(torch.int32).view(F32)
    else:
        top = bits.to(torch.int32).to(torch.uint16).view(dtype)
    x = torch.zeros(rows, cols, dtype=dtype)
    x[:32, :65536] = top
    x[:32, 65536:131072] = top.flip(1)
    g = torch.Generator().manual_seed(2)
    edges = torch.tensor([.25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 0.0, -0.0])
    below = edges[torch.randint(0, 16, (rows - 32, cols), generator=g)]
    below = below * torch.where(torch.rand(below.shape, generator=g) < 0.5, -1.0, 1.0)
    powers = torch.exp2(torch.randint(-14, 12, (rows - 32, 1), generator=g).float())
    x[32:] = (below * powers).to(dtype)
    x[32:, 64:96] = torch.finfo(dtype).smallest_normal * torch.rand(rows - 32, 32, generator=g).to(dtype)
    x[32:, 128:160] = 0.0
    x[32, 1000], x[rows - 1, 2001], x[32, cols - 1] = float("inf"), -float("inf"), float("nan")
    x[32, 5000] = torch.finfo(dtype).max
    return x


@by_type
@pytest.mark.parametrize("rows,cols", HEIGHTS[:2])
def test_quantize_every_value(rows, cols, dtype):
    assert quantize_height(rows, cols, MQ_TYPE[dtype], False, False) == (8 if dtype == F32 else 32)
    x = special(rows, cols, dtype)
    row, col = mq.MX4.empty(rows, cols), mq.MX4.empty(cols, rows)
    mq.mq_mx4_quantize(x.cuda(), row, col)
    same(row, *ref.quantize(f64(x)))
    same(col, *ref.quantize(f64(x).T))


@pytest.mark.parametrize("m,f,height", [(130, 22001, 8), (70, 300, 4)])
@by_type
def test_gated_backward_stochastic(m, f, height, dtype):
    """All four draws of a gradient, of numbers that 4 bits do not hold: dg = 2 dh or -2 dh and du = 32 dh or 0
    are exact before their rounding, and the products are exact after it."""
    assert quantize_height(m, f, MQ_TYPE[dtype], True, True) == height
    k, seed = 70, 9 << 33 | 5
    gen = torch.Generator(device="cuda").manual_seed(m)
    # multiples of 1/8 below 6, a 6 in each block of rows and of columns: every scale is that of a 6
    dh = (torch.randint(-47, 48, (m, f), generator=gen, device="cuda") / 8.0).to(dtype)
    dh[::32] = 6.0
    dh[:, ::32] = -6.0
    g, u = (torch.full((m, f), v, dtype=dtype, device="cuda") for v in (32.0, 2.0))
    u[1::2] = -2.0
    zero = mq.MX4(k, f, *(torch.zeros_like(t) for t in (random_held(3, k, f).codes, random_held(3, k, f).scales)))
    x_col, w = random_held(2, k, m), random_held(3, k, f)
    ws, new = mq.mx4_gated_backward_workspace(m, f, k), lambda r: torch.full((r, k), 3.0, device="cuda")
    dx_g, dx_u, dwg, dwu = new(m), new(m), new(f), new(f)
    mq.mq_mx4_gated_backward(dh, g, u, x_col, w, zero, dx_g, dwg, dwu, ws, mq.MQ_SR, seed)
    mq.mq_mx4_gated_backward(dh, g, u, None, zero, w, dx_u, None, None, ws, mq.MQ_SR, seed)
    dg, du = f64(dh) * f64(u), f64(dh) * 32.0
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    for got, v, d, q in ((dx_g, dg, 0, w), (dwg, dg.T, 1, x_col), (dx_u, du, 2, w), (dwu, du.T, 3, x_col)):
        rounded = ref.rounded(v, seed, d)
        assert not np.array_equal(rounded, v)
        assert torch.equal(got, product((cuda(rounded), values(q))).to(F32)), d


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("which", ["dh", "g", "u"])
def test_gated_backward_not_finite(which, bad):
    """One number that is not finite (a G or U past the range of f16, say) makes the sums of its row and of its
    column NaN, and no others."""
    m, f, k = 40, 70, 33
    t = {"dh": grid(1, m, f, F16, 0.25), "g": torch.full((m, f), 32.0, dtype=F16, device="cuda"),
         "u": torch.full((m, f), 2.0, dtype=F16, device="cuda")}
    t["dh"][t["dh"] == 0] = 0.5
    t[which][3, 65] = bad
    x_col, wg_col, wu_col = random_held(2, k, m), random_held(3, k, f), random_held(4, k, f)
    dx, dwg, dwu = (torch.empty(r, k, device="cuda") for r in (m, f, f))
    mq.mq_mx4_gated_backward(t["dh"], t["g"], t["u"], x_col, wg_col, wu_col, dx, dwg, dwu,
                             mq.mx4_gated_backward_workspace(m, f, k))
    rows = lambda n, *at: torch.tensor([i in at for i in range(n)], device="cuda")[:, None].expand(n, k)
    assert torch.equal(torch.isnan(dx), rows(m, 3)) and torch.isfinite(dx[4:]).all()
    assert torch.equal(torch.isnan(dwg), rows(f, 65)) and torch.isfinite(dwg[:65]).all()
    assert torch.equal(torch.isnan(dwu), rows(f, *([] if which == "u" else [65])))
