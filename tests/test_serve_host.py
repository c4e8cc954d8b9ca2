"""The serving layer's book-keeping (pages, lengths, refusals) on the CPU, its four calls replaced by
recorders."""
import pytest
import torch

import microscaling_quantized_convolution_amd as mq
from microscaling_quantized_convolution_amd import serve


@pytest.fixture
def calls(monkeypatch):
    """Names of the calls made, in order; a call named in `calls.refused` is refused."""
    class Calls(list):
        refused = None

    made = Calls()

    def record(name):
        def call(*args):
            if made.refused == name:
                raise mq.MQError(mq.MQ_ERR_ARG, name)
            made.append((name, args))
        return call
    for name in ("mq_attn_prompt", "mq_kv_append", "mq_attn_cached", "mq_kv_evict"):
        monkeypatch.setattr(serve, name, record(name))
    return made


def new_layer(n=2, max_len=64, page=16, num_pages=None):
    return serve.CachedAttention(n, max_len, 2, 1, 64, page, num_pages=num_pages, device="cpu")


def rows(tokens, heads, dim=64):
    return torch.zeros(tokens, heads, dim, dtype=torch.bfloat16)


def filled(layer, lengths):
    total = sum(lengths)
    layer.prefill(rows(total, 2), rows(total, 1), rows(total, 1), lengths)
    return layer


def state(layer):
    return (sorted(layer.free), [list(p) for p in layer.pages], list(layer.held), layer.lens.tolist(),
            layer.table.tolist())


def test_a_refused_eviction_changes_nothing(calls):
    layer = filled(new_layer(num_pages=12), [40, 20])
    before = state(layer)
    calls.refused = "mq_kv_evict"
    with pytest.raises(mq.MQError):
        layer.evict(16, 4)
    assert state(layer) == before
    calls.refused = None
    for keep, recent in ((-1, 0), (16, -1)):
        with pytest.raises(ValueError):
            layer.evict(keep, recent)
        assert state(layer) == before
    layer.evict(16, 4)
    assert layer.held == [16, 16] and len(layer.free) == 12 - 2
