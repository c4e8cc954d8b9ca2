"""GPU tests of the microscaled 4-bit layers at sizes that reach every way of the launches (rows, tiles
of every size, tall and short register tiles of the quantization), on other streams, in graphs, past
32-bit offsets. Large results are checked at rows and columns drawn from all of them."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_amd as mq
import mx4_reference as ref
from test_gpu_mx4 import BF16, F16, F32, dense, f64, held, random_codes, same

pytestmark = pytest.mark.gpu


def some(n, count=24, seed=0):
    """Numbers below n: the first, the last, those around multiples of 256, others."""
    rng = np.random.default_rng(seed)
    near = [b + d for b in range(0, n, max(256, n // 1024 * 256)) for d in (-1, 0)]
    pick = {0, n - 1, *rng.integers(0, n, count).tolist(), *rng.permutation(near)[:count].tolist()}
    return sorted(i for i in pick if 0 <= i < n)


def rows_of(q, rows):
    """Codes (bytes) and scales of some rows of a matrix on the GPU: [pieces][rows][...] on the CPU."""
    at = torch.tensor(rows, device="cuda")
    return q.codes[:, at].cpu(), q.scales[:, at].cpu()


def check_rows(q, rows, code, e):
    codes, scales = ref.packed(code, e)
    got = rows_of(q, rows)
    assert torch.equal(got[1], scales) and torch.equal(got[0], codes)


def spread(seed, rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") *
            torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))).to(dtype)


@pytest.mark.parametrize("sr", [None, 31], ids=["nearest", "stochastic"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(2100, 7300), (1000, 5001), (4099, 1111), (70, 66000)])
def test_quantize_many_tiles(rows, cols, dtype, sr):
    x = spread(rows, rows, cols, dtype)
    row, col = mq.MX4.empty(rows, cols), mq.MX4.empty(cols, rows)
    mq.mq_mx4_quantize(x, row, col, mq.MQ_RNE if sr is None else mq.MQ_SR, sr or 0)
    alone = mq.MX4.empty(rows, cols)
    mq.mq_mx4_quantize(x, alone, None, mq.MQ_RNE if sr is None else mq.MQ_SR, sr or 0)
    assert torch.equal(alone.codes, row.codes) and torch.equal(alone.scales, row.scales)
    if sr is None:
        at = some(rows)
        check_rows(row, at, *ref.quantize(f64(x[at])))
        at = some(cols)
        check_rows(col, at, *ref.quantize(f64(x[:, at]).T))
    else:  # draws go by the whole matrix
        same(row, *ref.quantize(f64(x), sr, 0))


@pytest.mark.parametrize("rows,cols,dtype", [(3000, 6001, F32), (5000, 6912, BF16), (16, 40, F16)])
def test_dequantize_large(rows, cols, dtype):
    q = random_held(rows, rows, cols)
    out = torch.full((rows + 1, cols + 3), 7.0, dtype=dtype, device="cuda")
    mq.mq_mx4_dequantize(q, out[:rows, 1:cols + 1])
    at = some(rows)
    assert torch.equal(out[at, 1:cols + 1].cpu(), torch.from_numpy(values_of(q, at)).to(dtype))
    assert (out[rows] == 7.0).all() and (out[:, 0] == 7.0).all() and (out[:, cols + 1:] == 7.0).all()


def random_held(seed, rows, cols):
    """A quantized matrix on the GPU of random codes, scales of [126, 128], and some of its rows' values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pieces = -(-cols // 256)
    codes = torch.randint(0, 256, (pieces, rows, 128), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(126, 129, (pieces, rows, 8), generator=g, device="cuda", dtype=torch.uint8)
    used = cols - (pieces - 1) * 256
    codes[-1, :, (used + 1) // 2:] = 0
    if used % 2:
        codes[-1, :, used // 2] &= 15
    return mq.MX4(rows, cols, codes, scales)


def values_of(q, rows):
    codes, scales = rows_of(q, rows)
    c = codes.permute(1, 0, 2).reshape(len(rows), -1).numpy()
    code = np.stack([c & 15, c >> 4], 2).reshape(len(rows), -1).astype(np.int64)
    e = scales.permute(1, 0, 2).reshape(len(rows), -1).numpy().astype(np.int64)
    return ref.values(code, e, q.shape[1])


@pytest.mark.parametrize("m,n,k", [(16, 12300, 700), (1, 20000, 300), (1100, 2900, 500), (2050, 3000, 300),
                                   (4000, 8230, 2049), (8200, 4100, 1900), (20000, 129, 300), (3, 12287, 4096),
                                   (640, 3300, 8192)])
def test_matmul_all_ways(m, n, k):
    """Sums of multiples of 2^-4 below 2^20: exact in fp32."""
    a, b = random_held(m, m, k), random_held(n + 1, n, k)
    y = torch.full((m, n), float("nan"), device="cuda")
    mq.mq_mx4_matmul(a, b, y, mq.mx4_matmul_workspace(m, n, k))
    at, to = some(m), some(n)
    want = values_of(a, at) @ values_of(b, list(range(n))).T
    assert np.abs(want).max() < 2.0 ** 20
    assert torch.equal(y[at].cpu(), torch.from_numpy(want).to(F32))
    want = values_of(a, list(range(m))) @ values_of(b, to).T
    assert torch.equal(y[:, to].cpu(), torch.from_numpy(want).to(F32))


@pytest.mark.parametrize("m,f,k", [(9, 13000, 300), (1000, 1500, 700), (2300, 1600, 300), (4100, 4000, 2049), (5, 11000, 4096)])
def test_gated_all_ways(m, f, k):
    x, wg, wu = spread(1, m, k, BF16), random_held(2, f, k), random_held(3, f, k)
    wg.scales -= 5
    h, g, u = (torch.full((m, f), float("nan"), device="cuda") for _ in range(3))
    mq.mq_mx4_gated(x, wg, wu, h, mq.mx4_gated_workspace(m, f, k), g, u)
    at = some(m)
    xq = ref.rounded(f64(x[at]))
    (rg, bg), (ru, bu) = (ref.product(xq, values_of(w, list(range(f)))) for w in (wg, wu))
    assert (np.abs(f64(g[at]) - rg) <= bg).all() and (np.abs(f64(u[at]) - ru) <= bu).all()
    assert not torch.isnan(g).any() and not torch.isnan(u).any() and not torch.isnan(h).any()
    # h from the very sums that were kept: the activation's own operations (as in test_gated)
    kg, ku = f64(g), f64(u)
    want = kg * ref.sigmoid(kg) * ku
    tiny = np.abs(ku) * 2.0 ** -100 + 2.0 ** -126  # exponentials past the range of fp32
    assert (np.abs(f64(h) - want) <= np.abs(want) * (16 * 2.0 ** -23 + np.minimum(np.abs(kg), 200) * 2.0 ** -22) + tiny).all()


@pytest.mark.parametrize("m,f,k", [(8200, 1100, 4096), (300, 5000, 130), (2100, 3000, 64)])
def test_gated_backward_all_ways(m, f, k):
    dh, g, u = (spread(s, m, f, BF16) for s in range(3))
    x_col, wg, wu = random_held(4, k, m), random_held(5, k, f), random_held(6, k, f)
    dx = torch.full((m, k), float("nan"), device="cuda")
    dwg, dwu = (torch.full((f, k), float("nan"), device="cuda") for _ in range(2))
    mq.mq_mx4_gated_backward(dh, g, u, x_col, wg, wu, dx, dwg, dwu, mq.mx4_gated_backward_workspace(m, f, k))

    def parts(pick, transpose):
        dhv, gv, uv = (f64(t[pick] if not transpose else t[:, pick].t()) for t in (dh, g, u))
        s = ref.sigmoid(gv)
        offs = np.abs(dhv * uv) * ref.LOOSE, np.abs(dhv * gv * s) * ref.LOOSE
        return zip(ref.gradients(dhv, gv, uv), offs)

    def part(v, off, w):
        want, bound = ref.product(ref.rounded(v), w)
        return want, bound + ref.unsure(v, off) @ np.abs(w).T
    at = some(m, 8)
    (a, ba), (b, bb) = (part(v, off, values_of(w, list(range(k)))) for (v, off), w in zip(parts(at, False), (wg, wu)))
    assert (np.abs(f64(dx[at]) - a - b) <= 2 * (ba + bb)).all()
    at = some(f, 8)
    xv = values_of(x_col, list(range(k)))
    for got, (v, off) in zip((dwg, dwu), parts(at, True)):
        want, bound = part(v, off, xv)
        assert (np.abs(f64(got[at]) - want) <= bound).all()


def test_offsets_past_32_bits():
    """Codes of more than 2^32 bytes, and outputs of more than 2^32 elements."""
    m, k = 600_000, 16384
    x = torch.randn(1200, k, device="cuda").bfloat16().repeat(m // 1200, 1)
    x[-1] *= 3.0
    row = mq.MX4.empty(m, k)
    mq.mq_mx4_quantize(x, row)
    at = [0, 1199, 1200, m // 2 + 7, m - 1201, m - 2, m - 1]
    check_rows(row, at, *ref.quantize(f64(x[at])))
    col = mq.MX4.empty(k, m)
    mq.mq_mx4_quantize(x, None, col)
    last = slice(m - m % 256 - 256, m)  # the last pieces of some columns
    code, e = ref.quantize(f64(x[last, [0, k // 2, k - 1]]).T)
    codes, scales = ref.packed(code, e)
    at_col = torch.tensor([0, k // 2, k - 1], device="cuda")
    pieces = codes.shape[0]
    assert torch.equal(col.codes[-pieces:][:, at_col].cpu(), codes) and torch.equal(col.scales[-pieces:][:, at_col].cpu(), scales)
    del x, col
    b = random_held(1, 24, k)
    y = torch.full((m, 24), float("nan"), device="cuda")
    mq.mq_mx4_matmul(row, b, y, mq.mx4_matmul_workspace(m, 24, k))
    want, bound = ref.product(values_of(row, at), values_of(b, list(range(24))))
    assert (np.abs(f64(y[at]) - want) <= bound).all() and not torch.isnan(y).any()
    del row, y
    n, k = 8000, 200
    a, b = random_held(2, m, k), random_held(3, n, k)
    y = torch.empty(m, n, dtype=BF16, device="cuda")
    mq.mq_mx4_matmul(a, b, y, mq.mx4_matmul_workspace(m, n, k))
    want = torch.from_numpy(values_of(a, at) @ values_of(b, list(range(n))).T).to(F32).to(BF16)
    assert torch.equal(y[at].cpu(), want)


def step(x, w, w_col, dy, ws, out):
    """A layer's forward and backward pass into the buffers of `out`."""
    mq.mq_mx4_linear(x, w, out["y"], ws, out["x_col"])
    mq.mq_mx4_linear_backward(dy, out["x_col"], w_col, out["dx"], out["dw"], ws, mq.MQ_SR, 5)


def step_buffers(m, n, k):
    z = lambda *s: torch.zeros(*s, dtype=BF16, device="cuda")
    return {"y": z(m, n), "x_col": mq.MX4.empty(k, m), "dx": z(m, k), "dw": z(n, k)}


def test_streams_and_graphs():
    """The same bits on another stream, and from two graphs replayed with other work between."""
    m, n, k = 200, 700, 600
    w = dense(3, n, k).cuda()
    w_row, w_col = mq.MX4.empty(n, k), mq.MX4.empty(k, n)
    mq.mq_mx4_quantize(w, w_row, w_col)
    sizes = max(mq.mx4_linear_workspace(m, n, k).numel(), mq.mx4_linear_backward_workspace(m, n, k).numel())
    ws = torch.empty(sizes, dtype=torch.uint8, device="cuda")
    inputs = [(dense(s, m, k, BF16).cuda(), dense(s + 10, m, n, BF16).cuda()) for s in range(2)]
    want = []
    for x, dy in inputs:
        out = step_buffers(m, n, k)
        step(x, w_row, w_col, dy, ws, out)
        want.append({key: out[key].clone() for key in ("y", "dx", "dw")})
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = step_buffers(m, n, k)
        step(inputs[0][0], w_row, w_col, inputs[0][1], ws, out)
    side.synchronize()
    assert all(torch.equal(out[key], want[0][key]) for key in want[0])
    out = step_buffers(m, n, k)  # a stream named in the call
    torch.cuda.synchronize()
    mq.mq_mx4_linear(inputs[0][0], w_row, out["y"], ws, out["x_col"], stream=side)
    side.synchronize()
    assert torch.equal(out["y"], want[0]["y"])
    # two graphs on one workspace, one after the other
    graphs, outs = [], []
    x, dy = inputs[0][0].clone(), inputs[0][1].clone()
    for _ in range(2):
        o, g = step_buffers(m, n, k), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(x, w_row, w_col, dy, ws, o)
        graphs.append(g)
        outs.append(o)
    for i in (0, 1, 0, 1, 1):
        x.copy_(inputs[i][0])
        dy.copy_(inputs[i][1])
        for g, o in zip(graphs, outs):
            g.replay()
            ws.fill_(0xAB)  # a workspace holds nothing from call to call
            torch.cuda.synchronize()
            assert all(torch.equal(o[key], want[i][key]) for key in want[i])
            step(inputs[1 - i][0], w_row, w_col, inputs[1 - i][1], ws, step_buffers(m, n, k))


def test_binding_refusals():
    z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")
    x, y, w = z(4, 64), z(4, 32), mq.MX4.empty(32, 64)
    ws = mq.mx4_linear_workspace(4, 32, 64)
    for bad in (z(64, 4).t(), z(4), z(4, 64, 1), z(4, 64, dtype=torch.float64), z(4, 64).cpu(),
                z(1, 64).expand(4, 64)):
        with pytest.raises(ValueError, match="x:"):
            mq.mq_mx4_linear(bad, w, y, ws)
    for bad in (z(4, 33), z(5, 32)):
        with pytest.raises(mq.MQError):
            mq.mq_mx4_linear(x, w, bad, ws)
    with pytest.raises(mq.MQError):
        mq.mq_mx4_linear(x, w, y, None)
    with pytest.raises(mq.MQError):
        mq.mq_mx4_linear(x, w, y, ws[:-1])
    with pytest.raises(ValueError, match="ws"):
        mq.mq_mx4_linear(x, w, y, ws.cpu())
    with pytest.raises(ValueError, match="codes"):
        mq.MX4(32, 64, w.codes[:, :-1], w.scales)
    with pytest.raises(ValueError, match="scales"):
        mq.MX4(32, 64, w.codes, w.scales.float())
    with pytest.raises(mq.MQError):
        mq.mq_mx4_quantize(x, None, None)
    with pytest.raises(mq.MQError):
        mq.mq_mx4_quantize(x, mq.MX4.empty(64, 4))
    with pytest.raises(mq.MQError):
        mq.mq_mx4_quantize(x, mq.MX4.empty(4, 64), rnd=2)
    with pytest.raises(ValueError, match="current device"):
        mq.mq_mx4_quantize(x, mq.MX4.empty(4, 64, "cpu"))
    with pytest.raises(ValueError, match="sizes"):
        mq.mx4_gated_workspace(-1, 3, 4)
    assert mq.mq_mx4_matmul(w, mq.MX4.empty(5, 64), z(32, 5)) is None


@pytest.mark.parametrize("m,f,k", [(7, 100, 300), (70, 333, 257), (700, 1300, 520)])
def test_gated_views(m, f, k):
    """Inputs and outputs inside larger matrices, rows of any alignment, one weight in both places: the
    same bits as from matrices of their own, and nothing written around the outputs."""
    def inside(t, fill=3.0):
        big = torch.full((t.shape[0] + 3, t.shape[1] + 13), fill, dtype=t.dtype, device="cuda")
        view = big[2:2 + t.shape[0], 5:5 + t.shape[1]]
        view.copy_(t)
        return big, view
    x, dh = spread(1, m, k, BF16), spread(2, m, f, BF16)
    w, w_col, x_col = random_held(3, f, k), random_held(4, k, f), mq.MX4.empty(k, m)
    w.scales -= 4
    ws = torch.empty(max(mq.mx4_gated_workspace(m, f, k).numel(), mq.mx4_gated_backward_workspace(m, f, k).numel()),
                     dtype=torch.uint8, device="cuda")
    new = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")
    out = {"h": new(m, f), "g": new(m, f), "u": new(m, f), "dx": new(m, k), "dwg": new(f, k, dtype=F32),
           "dwu": new(f, k, dtype=F32)}

    def run(x, dh, o):
        mq.mq_mx4_gated(x, w, w, o["h"], ws, o["g"], o["u"], x_col)
        mq.mq_mx4_gated_backward(dh, o["g"], o["u"], x_col, w_col, w_col, o["dx"], o["dwg"], o["dwu"], ws)
    run(x, dh, out)
    assert torch.equal(out["g"], out["u"])
    views = {name: inside(torch.zeros_like(t)) for name, t in out.items()}
    run(inside(x, float("nan"))[1], inside(dh, float("nan"))[1], {name: v[1] for name, v in views.items()})
    for name, (big, view) in views.items():
        assert torch.equal(view, out[name]), name
        view.fill_(3.0)
        assert (big == 3.0).all(), name


def test_two_streams_at_once():
    """Calls side by side on two streams, each with its own workspace: the bits of each alone."""
    m, f, k = 900, 1500, 700
    wg, wu = random_held(1, f, k), random_held(2, f, k)
    xs = [spread(s, m, k, BF16) for s in range(2)]
    want = []
    for x in xs:
        want.append(torch.empty(m, f, dtype=BF16, device="cuda"))
        mq.mq_mx4_gated(x, wg, wu, want[-1], mq.mx4_gated_workspace(m, f, k))
    streams, got = [torch.cuda.Stream() for _ in xs], [torch.zeros_like(w) for w in want]
    spaces = [mq.mx4_gated_workspace(m, f, k) for _ in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, y, ws, st in zip(xs, got, spaces, streams):
            mq.mq_mx4_gated(x, wg, wu, y, ws, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
