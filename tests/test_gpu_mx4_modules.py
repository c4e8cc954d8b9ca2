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


class Calls:
    """The library's calls as a module makes them: names, and which outputs beside the first are asked for."""

    def __init__(self, monkeypatch):
        self.made = []
        for name in ("mq_mx4_linear", "mq_mx4_gated", "mq_mx4_quantize"):
            monkeypatch.setattr(mqnn, name, self.watch(name, getattr(mqnn, name)))

    def watch(self, name, call):
        def made(*args):
            extra = args[{"mq_mx4_linear": 4, "mq_mx4_gated": 5, "mq_mx4_quantize": 2}[name]:]
            self.made.append((name, any(isinstance(a, (torch.Tensor, mq.MX4)) for a in extra)))
            return call(*args)
        return made


@pytest.mark.parametrize("tokens", [1, 40])
@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_no_training_work_without_a_graph(monkeypatch, mode, tokens):
    """Where no graph is recorded, nothing is made for a backward pass: neither the input's columns nor the
    weight's, nor the two projections; with weights held, a call makes the products alone."""
    m, x = block(), dense(1, tokens, 64, BF16).cuda()
    want = m(x).detach()
    lone = mqnn.MXLinear(64, 33).cuda()
    with mode():
        m(x)
        calls = Calls(monkeypatch)
        assert torch.equal(m(x), want)
        assert calls.made == [("mq_mx4_gated", False), ("mq_mx4_linear", False)]
        calls.made.clear()
        lone(x)  # a module in training, as in an evaluation between steps
        assert calls.made == [("mq_mx4_quantize", False), ("mq_mx4_linear", False)]
    calls.made.clear()
    m(x)  # and with a graph, for the weights
    assert ("mq_mx4_gated", True) in calls.made and ("mq_mx4_linear", True) in calls.made
