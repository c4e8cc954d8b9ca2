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
