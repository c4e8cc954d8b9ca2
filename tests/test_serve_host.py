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


def evicted(calls):
    """Lengths of the sequences in each eviction that was made."""
    return [args[2].tolist() for name, args in calls if name == "mq_kv_evict"]


@pytest.mark.parametrize("n,keep", [(8, 1024), (3, 2048), (1, 4095), (5, 0)])
def test_a_full_layer_of_the_default_size_can_evict(calls, n, keep):
    """Every sequence at max_len: nothing more can be appended, and a cut fits the pool."""
    full, page = 4096, 64
    layer = filled(new_layer(n, full, page), [full] * n)
    with pytest.raises(ValueError):
        layer.decode(rows(n, 2), rows(n, 1), rows(n, 1))
    pool = layer.cache.num_pages
    layer.evict(keep, 0)
    assert layer.held == [keep] * n == layer.lens.tolist()
    assert sorted(sum(layer.pages, []) + layer.free) == list(range(pool))
    assert [len(p) for p in layer.pages] == [-(-keep // page)] * n
    for p, row in zip(layer.pages, layer.table.tolist()):
        assert row == p + [-1] * (len(row) - len(p))
    assert sum(evicted(calls), []) == [full] * n  # each of them once
    assert layer.positions.shape == (n, 1, keep)
    layer.decode(rows(n, 2), rows(n, 1), rows(n, 1))


def test_an_eviction_with_room_is_one_call(calls):
    layer = filled(new_layer(4, 64, 16, num_pages=64), [64] * 4)
    layer.evict(32, 8)
    assert evicted(calls) == [[64] * 4]


def test_short_sequences_stay_where_they_are(calls):
    layer = filled(new_layer(3, 64, 16), [64, 20, 33])
    kept = list(layer.pages[1])
    layer.evict(32, 8)
    assert evicted(calls) == [[64, 33]] and layer.pages[1] == kept
    assert layer.held == [32, 20, 32] == layer.lens.tolist()
    assert layer.positions[1, 0].tolist() == list(range(20)) + [-1] * 12


def test_an_eviction_without_room_changes_nothing(calls):
    layer = filled(new_layer(2, 64, 16, num_pages=8), [64, 64])
    before = state(layer)
    with pytest.raises(RuntimeError):
        layer.evict(32, 8)
    assert state(layer) == before and not evicted(calls)


def test_an_eviction_refused_half_way_keeps_what_was_done(calls, monkeypatch):
    layer = filled(new_layer(3, 64, 16), [64] * 3)  # 4 free pages: two sequences at a time
    call = serve.mq_kv_evict

    def second_refused(*args):
        if evicted(calls):
            calls.refused = "mq_kv_evict"
        call(*args)
    monkeypatch.setattr(serve, "mq_kv_evict", second_refused)
    with pytest.raises(mq.MQError):
        layer.evict(32, 0)
    assert evicted(calls) == [[64, 64]] and layer.held == [32, 32, 64] == layer.lens.tolist()
    assert sorted(sum(layer.pages, []) + layer.free) == list(range(16))
    assert [len(p) for p in layer.pages] == [2, 2, 4]
    for p, row in zip(layer.pages, layer.table.tolist()):
        assert row == p + [-1] * (len(row) - len(p))


@pytest.mark.parametrize("lengths,tokens", [([40, 20], (59, 60, 60)), ([40, 20], (60, 61, 60)),
                                            ([40, 20], (60, 60, 59)), ([60], (60, 60, 60)),
                                            ([20, 20, 20], (60, 60, 60)), ([70, -10], (60, 60, 60))])
def test_prefill_refuses_lengths_that_do_not_fit(calls, lengths, tokens):
    """Before anything is launched or changed: a length for each sequence, none negative, and as
    many rows as they add up to."""
    layer = new_layer(max_len=128)
    before = state(layer)
    with pytest.raises(ValueError):
        layer.prefill(rows(tokens[0], 2), rows(tokens[1], 1), rows(tokens[2], 1), lengths)
    assert not calls and state(layer) == before


def test_a_refused_step_can_be_made_again(calls):
    """A step whose attention is refused has added no token."""
    layer = filled(new_layer(), [16, 5])
    calls.refused = "mq_attn_cached"
    for _ in range(2):
        with pytest.raises(mq.MQError):
            layer.decode(rows(2, 2), rows(2, 1), rows(2, 1))
        assert layer.held == [16, 5] == layer.lens.tolist()
    calls.refused = None
    layer.decode(rows(2, 2), rows(2, 1), rows(2, 1))
    assert layer.held == [17, 6] == layer.lens.tolist() and calls[-1][1][3].tolist() == [17, 6]
    assert sorted(sum(layer.pages, []) + layer.free) == list(range(layer.cache.num_pages))


def test_a_step_is_sized_by_the_longest_sequence(calls):
    """Not by what the layer could hold: grid and scratch of the attention go by its max_len."""
    layer = filled(new_layer(max_len=1 << 17, num_pages=64, page=64), [100, 30])
    need = lambda length: mq.mq_attn_cached_workspace_bytes(2, 2, 1, 64, 1, length, True)
    for longest in range(101, 140):
        layer.decode(rows(2, 2), rows(2, 1), rows(2, 1))
        ws, max_len = calls[-1][1][5], calls[-1][1][8]
        assert max_len == longest == max(layer.held)
        assert need(longest) <= ws.numel() <= need(2 * longest)
