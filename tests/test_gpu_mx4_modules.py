"""GPU tests of what the 4-bit modules keep from one call to the next, and from the forward pass to the
backward pass: copies, other streams, captured graphs, weights that change, memory."""
import copy
import io
import pickle

import pytest
import torch

import microscaling_quantized_convolution_amd as mq
from microscaling_quantized_convolution_amd import nn as mqnn
from microscaling_quantized_convolution_amd import serve
from test_gpu_mx4 import BF16, F16, F32, dense

pytestmark = pytest.mark.gpu


def block(features=64, hidden=96, **more):
    torch.manual_seed(5)
    return mqnn.MXGatedMLP(features, hidden, cache_weight=True, **more).cuda().eval()


def fresh(module, x):
    """The module's outputs from its parameters as they are now."""
    with torch.no_grad():
        h = mqnn.MXGatedFunction.apply(x, module.gate, module.up, 0, None)
        return mqnn.MXLinearFunction.apply(h, module.down.weight, 0, None)


@pytest.mark.parametrize("way", [copy.deepcopy, lambda t: pickle.loads(pickle.dumps(t))], ids=["deepcopy", "pickle"])
def test_copies(way):
    m, x = block(), dense(1, 5, 64, BF16).cuda()
    with torch.no_grad():
        y = m(x)
        other = way(m)
        assert torch.equal(other(x), y)
        m.gate.mul_(2.0)
        assert torch.equal(other(x), y) and torch.equal(m(x), fresh(m, x))
    feed = serve.FeedForward(m.gate.detach(), m.up.detach(), m.down.weight.detach(), 8)
    want = feed(x)
    other = way(feed)
    feed.gate.codes.zero_()
    assert torch.equal(other(x), want) and not torch.equal(feed(x), want)


def test_saved_module():
    m, x = block(), dense(1, 5, 64, BF16).cuda()
    with torch.no_grad():
        y = m(x)
        file = io.BytesIO()
        torch.save(m, file)
        file.seek(0)
        assert torch.equal(torch.load(file, weights_only=False)(x), y)
