"""GPU tests of the modules and the serving block over the 4-bit layers: they make the library's calls
in the documented order (the same bits as by hand), train, run under graphs and refuse bad inputs."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_amd as mq
import mx4_reference as ref
from microscaling_quantized_convolution_amd import nn as mqnn
from microscaling_quantized_convolution_amd import serve
from test_gpu_mx4 import BF16, F16, F32, dense, f64

pytestmark = pytest.mark.gpu


def quantized(w, columns=True):
    row = mq.MX4.empty(*w.shape)
    col = mq.MX4.empty(w.shape[1], w.shape[0]) if columns else None
    mq.mq_mx4_quantize(w, row, col)
    return row, col


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(3, 5, 96), (70, 96), (96,)])
def test_linear_module(shape, dtype):
    layer = mqnn.MXLinear(96, 200, layer_index=2, layers=5, seed_base=11).cuda()
    x = torch.randn(*shape, device="cuda").to(dtype).requires_grad_()
    y = layer(x)
    assert y.shape == (*shape[:-1], 200) and y.dtype == dtype
    gy = torch.randn_like(y)
    y.backward(gy)
    rows, m = x.detach().reshape(-1, 96), x.numel() // 96
    w = layer.weight.detach()
    row, col = quantized(w)
    out, x_col = torch.empty(m, 200, dtype=dtype, device="cuda"), mq.MX4.empty(96, m)
    mq.mq_mx4_linear(rows, row, out, mq.mx4_linear_workspace(m, 200, 96), x_col)
    assert torch.equal(y.detach().view(m, 200), out)
    dx, dw = torch.empty_like(rows), torch.empty_like(w)
    mq.mq_mx4_linear_backward(gy.reshape(m, 200), x_col, col, dx, dw, mq.mx4_linear_backward_workspace(m, 200, 96),
                              mq.MQ_SR, 11 + 2)
    assert torch.equal(x.grad.view(m, 96), dx) and torch.equal(layer.weight.grad, dw)
    assert layer.step == 1
    # only what is asked for
    frozen = mqnn.MXLinear(96, 200).cuda().requires_grad_(False)
    z = x.detach().clone().requires_grad_()
    frozen(z).sum().backward()
    assert frozen.weight.grad is None and z.grad is not None
    layer.zero_grad()
    layer(x.detach()).sum().backward()
    assert layer.weight.grad is not None


def test_gated_module():
    """One block's step, by hand from the library's calls."""
    m, d, f = 60, 128, 300
    block = mqnn.MXGatedMLP(d, f, layer_index=1, layers=3, seed_base=7).cuda()
    x = torch.randn(m, d, device="cuda").bfloat16().requires_grad_()
    y = block(x)
    gy = torch.randn_like(y)
    y.backward(gy)
    (wg, wg_col), (wu, wu_col), (wd, wd_col) = (quantized(w.detach()) for w in (block.gate, block.up, block.down.weight))
    new = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="cuda")
    h, g, u, x_col = new(m, f), new(m, f), new(m, f), mq.MX4.empty(d, m)
    mq.mq_mx4_gated(x.detach(), wg, wu, h, mq.mx4_gated_workspace(m, f, d), g, u, x_col)
    out, h_col = new(m, d), mq.MX4.empty(f, m)
    mq.mq_mx4_linear(h, wd, out, mq.mx4_linear_workspace(m, d, f), h_col)
    assert torch.equal(out, y.detach())
    dh, dwd = new(m, f), new(d, f, dtype=F32)
    mq.mq_mx4_linear_backward(gy, h_col, wd_col, dh, dwd, mq.mx4_linear_backward_workspace(m, d, f), mq.MQ_SR, 7 + 3)
    dx, dwg, dwu = new(m, d), new(f, d, dtype=F32), new(f, d, dtype=F32)
    mq.mq_mx4_gated_backward(dh, g, u, x_col, wg_col, wu_col, dx, dwg, dwu, mq.mx4_gated_backward_workspace(m, f, d),
                             mq.MQ_SR, 7 + 2)
    for got, want in ((x.grad, dx), (block.gate.grad, dwg), (block.up.grad, dwu), (block.down.weight.grad, dwd)):
        assert torch.equal(got, want)
    # the next step draws other bits
    x2 = x.detach().clone().requires_grad_()
    block.zero_grad()
    block(x2).backward(gy)
    assert torch.equal(out, block.eval()(x.detach())) and not torch.equal(x2.grad, x.grad)


def test_gradients_are_those_of_the_products():
    """With inputs, weights and gradients that 4 bits hold exactly, nothing is rounded: gradients equal
    those of the plain layer in 64 bits."""
    g = torch.Generator().manual_seed(3)
    grid = torch.tensor([-6, -4, -3, -2, -1.5, -1, -.5, 0, .5, 1, 1.5, 2, 3, 4, 6])
    pick = lambda *s: grid[torch.randint(0, 15, s, generator=g)].index_fill(0, torch.tensor([0]), 6.0).index_fill(1, torch.arange(0, s[1], 32), 6.0)
    # every 32 of a row or of a column holds a 6, so that all scales are 1
    full = lambda *s: pick(*s).index_fill(0, torch.arange(0, s[0], 32), 6.0)
    x, w, gy = full(64, 96), full(128, 96), full(64, 128)
    layer = mqnn.MXLinear(96, 128).cuda()
    with torch.no_grad():
        layer.weight.copy_(w)
    xg = x.cuda().requires_grad_()
    layer(xg).backward(gy.cuda())
    a, b = x.double().requires_grad_(), w.double().requires_grad_()
    (a @ b.t()).backward(gy.double())
    assert torch.equal(xg.grad.cpu().double(), a.grad) and torch.equal(layer.weight.grad.cpu().double(), b.grad)


def test_cached_weights():
    block = mqnn.MXGatedMLP(64, 96, cache_weight=True).cuda().eval()
    x = torch.randn(4, 64, device="cuda").half()
    with torch.no_grad():
        y = block(x)
        held = block._held
        assert torch.equal(block(x), y) and block._held is held
        block.gate.mul_(2.0)
        z = block(x)
    assert block._held is not held and not torch.equal(z, y)
    held = block._held
    with torch.no_grad():  # another parameter in the place of one, and the same one in other types
        block.up = torch.nn.Parameter(block.up.detach() * 3.0)
        assert not torch.equal(block(x), z) and block._held is not held
        held = block._held
        block.half()
        block(x)
        assert block._held is not held
        block.float()
    # a gradient with respect to the input still goes through held weights
    xr = x.clone().requires_grad_()
    block.requires_grad_(False)
    block(xr).sum().backward()
    assert xr.grad is not None and torch.isfinite(xr.grad).all()


def test_module_refusals():
    layer = mqnn.MXLinear(64, 32).cuda()
    for bad in (torch.zeros(4, 64), torch.zeros(4, 63, device="cuda"), torch.zeros(4, 64, device="cuda").double()):
        with pytest.raises(ValueError):
            layer(bad)
    assert layer(torch.zeros(0, 64, device="cuda")).shape == (0, 32)


@pytest.mark.parametrize("tokens", [1, 3, 16, 17, 100])
def test_feed_forward(tokens):
    d, f = 256, 700
    gate, up, down = (dense(s, *shape).cuda() / 16 for s, shape in ((1, (f, d)), (2, (f, d)), (3, (d, f))))
    feed = serve.FeedForward(gate, up, down, 100)
    big = torch.randn(tokens, d + 8, device="cuda").bfloat16()
    x = big[:, 8:]
    y = feed(x)
    xq, g, u, w = ref.rounded(f64(x)), *(ref.rounded(f64(t)) for t in (gate, up, down))
    rg, ru = xq @ g.T, xq @ u.T
    h = torch.from_numpy(rg * ref.sigmoid(rg) * ru)
    # h is rounded to bf16 and then to 4 bits: what lies next to a border may fall to either side
    off = np.abs(h.numpy()) * 2.0 ** -8 + 1e-6
    want, bound = ref.product(ref.rounded(h.to(F32).to(BF16).double().numpy()), w)
    bound = bound + ref.unsure(h.numpy(), off) @ np.abs(w).T
    assert (np.abs(f64(y) - want) <= bound + ref.half_step(BF16, np.abs(want) + bound)).all()
    block = mqnn.MXGatedMLP(d, f).cuda().eval()
    with torch.no_grad():
        block.gate.copy_(gate), block.up.copy_(up), block.down.weight.copy_(down)
        assert torch.equal(block(x), y)
    g = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(g):
        out = feed(xs)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)


def test_feed_forward_refusals():
    gate, down = torch.zeros(64, 32, device="cuda"), torch.zeros(32, 64, device="cuda")
    with pytest.raises(ValueError, match="down"):
        serve.FeedForward(gate, gate, gate, 4)
    with pytest.raises(ValueError, match="max_tokens"):
        serve.FeedForward(gate, gate, down, 0)
    feed = serve.FeedForward(gate, gate, down, 4)
    for bad in (torch.zeros(5, 32, device="cuda"), torch.zeros(4, 33, device="cuda"), torch.zeros(32, device="cuda")):
        with pytest.raises(ValueError, match="expected up to 4 rows"):
            feed(bad)
    assert feed(torch.zeros(0, 32, device="cuda")).shape == (0, 32)


def test_attention_and_feed_forward_together():
    """A decoder layer's serving steps: prompts, then tokens, each through the attention and the block."""
    n, q_heads, heads, dim, lengths = 2, 4, 2, 64, [37, 5]
    width = q_heads * dim
    layer = serve.CachedAttention(n, 96, q_heads, heads, dim, 32)
    feed = serve.FeedForward(*(dense(s, *shape).cuda() / 16 for s, shape in ((1, (512, width)), (2, (512, width)),
                                                                              (3, (width, 512)))), sum(lengths))
    new = lambda tokens, h: torch.randn(tokens, h, dim, device="cuda").bfloat16()
    total = sum(lengths)
    out = layer.prefill(new(total, q_heads), new(total, heads), new(total, heads), lengths)
    y = feed(out.view(total, width))
    h, by_hand = torch.empty(total, 512, dtype=BF16, device="cuda"), torch.empty_like(y)
    mq.mq_mx4_gated(out.view(total, width), feed.gate, feed.up, h, mq.mx4_gated_workspace(total, 512, width))
    mq.mq_mx4_linear(h, feed.down, by_hand, mq.mx4_linear_workspace(total, width, 512))
    assert torch.equal(by_hand, y)
    for _ in range(3):
        step = layer.decode(new(n, q_heads), new(n, heads), new(n, heads))
        assert torch.isfinite(feed(step.view(n, width))).all()
