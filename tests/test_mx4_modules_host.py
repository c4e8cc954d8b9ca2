"""What the 4-bit modules and matrices promise without a GPU: copies and pickles, and seeds."""
import copy
import io
import pickle

import pytest
import torch

import microscaling_quantized_convolution_amd as mq
from microscaling_quantized_convolution_amd import nn as mqnn


def matrix(rows, cols):
    q = mq.MX4.empty(rows, cols, "cpu")
    q.codes.random_(0, 256)
    q.scales.random_(2, 253)
    return q


def saved_and_loaded(thing):
    file = io.BytesIO()
    torch.save(thing, file)
    file.seek(0)
    return torch.load(file, weights_only=False)


@pytest.mark.parametrize("rows,cols", [(3, 300), (1, 1), (0, 40), (5, 0)])
@pytest.mark.parametrize("way", [copy.deepcopy, lambda q: pickle.loads(pickle.dumps(q)), saved_and_loaded],
                         ids=["deepcopy", "pickle", "save"])
def test_matrix_copies(way, rows, cols):
    q = matrix(rows, cols)
    p = way(q)
    assert p.shape == q.shape and torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
    # its structure points into its own tensors, not into the first one's
    assert (p.struct.codes or 0) == p.codes.data_ptr() and (p.struct.scales or 0) == p.scales.data_ptr()
    if q.codes.numel():
        before = p.codes.clone()
        q.codes.bitwise_not_()
        assert torch.equal(p.codes, before)


def test_matrix_shared_copy():
    """copy.copy shares the tensors, as it does for other objects; one matrix held twice stays one."""
    q = matrix(2, 70)
    assert copy.copy(q).codes is q.codes
    a, b = copy.deepcopy([q, q])
    assert a is b and a is not q


def model():
    """Projections, gated blocks and a convolution in one model, each number given as if all were of one kind."""
    parts = [mqnn.MXLinear(32, 32, i, 6, 9) for i in (0, 1, 3, 4)]
    parts[2:2] = [mqnn.MXGatedMLP(32, 64, 2, 6, 9)]
    return torch.nn.Sequential(*parts, mqnn.MXGatedMLP(32, 64, 5, 6, 9), mqnn.MQConv2d(4, 4, 3, layer_index=2, layers=6))


def seeds(m, steps):
    """The seeds of every gradient that the model's layers round, over some steps."""
    found = [p for p in m.modules() if hasattr(p, "layer_index")]
    drawn = []
    for _ in range(steps):
        for p in found:
            if isinstance(p, mqnn.MQConv2d):
                drawn.append(p.sr_seed())
                p.step += 1
            else:
                drawn.append(p._next_seed())
    return drawn


def test_seeds_of_a_mixed_model():
    """Numbered through, no two layers or steps share a seed, whatever their kinds; a model without gated
    blocks keeps the numbers that it would be given by hand."""
    m = model()
    assert mqnn.number_layers(m, 9) == 9
    drawn = seeds(m, 5)
    assert len(drawn) == 45 and sorted(drawn) == list(range(9, 54))
    net = mqnn.ResNet18MQ(fmt=mq.MQ_NVFP4, seed_base=4)
    before = [c.sr_seed() for c in net.mq_convs]
    assert mqnn.number_layers(net, 4) == len(before) and [c.sr_seed() for c in net.mq_convs] == before


def test_seeds_of_one_kind():
    """By hand: projections by their numbers, gated blocks by pairs of numbers."""
    for make, each in ((lambda i: mqnn.MXLinear(32, 32, i, 4, 3), 1), (lambda i: mqnn.MXGatedMLP(32, 32, i, 4, 3), 2)):
        m = torch.nn.Sequential(*(make(i) for i in range(4)))
        drawn = seeds(m, 3)
        assert sorted(drawn) == list(range(3, 3 + 12 * each))


def test_modules_pickle_without_held_weights():
    """A module's pickle has its parameters, numbers and steps alone, and one made without the rest is whole."""
    m = mqnn.MXGatedMLP(32, 64, 1, 3, 7, cache_weight=True)
    m.step, m.down.step = 4, 5
    m._kept = [object()], [], None, None
    other = pickle.loads(pickle.dumps(m))
    assert other._held is None and other.down._held is None and m._held is not None
    assert (other.step, other.down.step, other.cache_weight) == (4, 5, True)
    assert all(torch.equal(a, b) for a, b in zip(m.parameters(), other.parameters()))
    del other.__dict__["_kept"]
    assert other._held is None and other.eval()._held is None
    m.train()
    assert m._held is None
