"""The serving layer (prompts, new tokens, eviction) against the 64-bit definitions of its calls in
the same order, and the binding's refusals."""
import math

import pytest
import torch

import attn_reference as ref
import microscaling_quantized_convolution_amd as mq
from microscaling_quantized_convolution_amd import serve

pytestmark = pytest.mark.gpu


def test_layer_matches_reference():
    n, q_heads, heads, dim, page = 3, 4, 2, 64, 16
    lengths, scale = [70, 5, 33], 0.125
    gen = torch.Generator().manual_seed(1)
    new = lambda tokens, h: torch.randn(tokens, h, dim, generator=gen).bfloat16()
    layer = serve.CachedAttention(n, 96, q_heads, heads, dim, page, scale=scale)
    cache = ref.empty_cache(layer.cache.num_pages, page, heads, dim)
    weights = torch.zeros(layer.cache.weights_shape, dtype=torch.float64)
    slack = torch.zeros_like(weights)

    def table():
        return layer.table.tolist()

    q, k, v = new(sum(lengths), q_heads), new(sum(lengths), heads), new(sum(lengths), heads)
    out = layer.prefill(q.cuda(), k.cuda(), v.cuda(), lengths)
    cu = [sum(lengths[:i]) for i in range(n + 1)]
    want, bound = ref.prompt(q, k, v, cu, scale)
    assert ((out.cpu().double() - want).abs() <= bound).all()
    ref.append(cache, k, v, table(), [0] * n, cu)
    held = list(lengths)

    def decode():
        q, k, v = new(n, q_heads), new(n, heads), new(n, heads)
        out = layer.decode(q.cuda(), k.cuda(), v.cuda())
        ref.append(cache, k, v, table(), held, list(range(n + 1)))
        held[:] = [h + 1 for h in held]
        assert layer.held == held == layer.lens.tolist()
        want, bound, given, given_bound = ref.cached(cache, q, table(), held, 1, scale)
        assert ((out.cpu().double() - want).abs() <= bound).all()
        weights.add_(given)
        slack.add_(given_bound + 2.0 ** -23 * weights)

    for _ in range(13):
        decode()
    got = layer.weights.cpu().double()
    used = torch.zeros_like(weights, dtype=torch.bool)
    for row, h in zip(table(), held):
        for t in range(h):
            used[row[t // page], :, t % page] = True
    assert ((got - weights).abs() <= slack)[used].all()

    old, before = table(), layer.lens.tolist()
    layer.evict(24, 6)
    kept, new_lens = ref.evict(cache, layer_weights := got.float(), old, before,
                               [r[:2] for r in table()], 24, 6)
    assert layer.held == new_lens == layer.lens.tolist()
    assert layer.positions.tolist() == kept
    held[:] = new_lens
    weights.copy_(layer_weights.double())
    slack.zero_()
    for _ in range(3):
        decode()


def test_layer_pages():
    """Pages come back after an eviction; a layer that runs out says so and keeps its state."""
    layer = serve.CachedAttention(2, 64, 2, 1, 64, 16, num_pages=7)
    new = lambda tokens, h: torch.randn(tokens, h, 64, device="cuda").bfloat16()
    layer.prefill(new(60, 2), new(60, 1), new(60, 1), [40, 20])
    assert len(layer.free) == 7 - 3 - 2
    with pytest.raises(ValueError):
        layer.prefill(new(1, 2), new(1, 1), new(1, 1), [1, 0])
    layer.evict(16, 4)
    assert layer.held == [16, 16] and len(layer.free) == 5
    with pytest.raises(RuntimeError):
        layer.free.clear()
        layer.decode(new(2, 2), new(2, 1), new(2, 1))
    assert layer.held == [16, 16] == layer.lens.tolist()
    with pytest.raises(ValueError):
        layer._reserve([49, 0])


def test_fresh_pages_hold_no_weights():
    """Slots of a page behind the kept tokens start at weight 0, whoever had the page before."""
    layer = serve.CachedAttention(1, 128, 2, 1, 64, 64, num_pages=4)
    new = lambda tokens, h: torch.randn(tokens, h, 64, device="cuda").bfloat16()
    layer.weights.fill_(9.0)
    layer.prefill(new(100, 2), new(100, 1), new(100, 1), [100])
    layer.evict(20, 20)
    layer.decode(new(1, 2), new(1, 1), new(1, 1))
    w = layer.weights[layer.pages[0][0], 0]
    assert abs(w.sum().item() - 2.0) < 1e-4  # one new row of two heads, nothing else


def test_demo_runs(capsys):
    serve.main()
    assert "tokens held [65, 65, 65]" in capsys.readouterr().out


def test_binding_refuses():
    n, dim = 2, 64
    c = mq.KVCache.empty(4, 16, 2, dim)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    k = torch.zeros(3, 2, dim, dtype=torch.bfloat16, device="cuda")
    table, lens, cu = i32(*range(4)).view(2, 2), i32(0, 0), i32(0, 1, 3)
    mq.mq_kv_append(k, k, c, table, lens, cu)
    for args in ((k.float(), k, c, table, lens, cu), (k.cpu(), k, c, table, lens, cu),
                 (k[0], k, c, table, lens, cu), (k.transpose(1, 2), k, c, table, lens, cu),
                 (k, k, c, table.long(), lens, cu), (k, k, c, table[:1], lens, cu),
                 (k, k, c, table[:, ::2], lens, cu), (k, k, c, table.view(-1), lens, cu),
                 (k, k, c, table, lens.cpu(), cu), (k, k, c, table, lens, cu[:2])):
        with pytest.raises(ValueError):
            mq.mq_kv_append(*args)
    with pytest.raises(mq.MQError) as e:  # refused by the library
        mq.mq_kv_append(k[:2], k, c, table, lens, cu)
    assert e.value.status == mq.MQ_ERR_SHAPE
    q, out = k[:2], torch.empty_like(k[:2])
    w = torch.zeros(c.weights_shape, device="cuda")
    ws = mq.attn_cached_workspace(n, 2, 2, dim, 1, 32, True)
    mq.mq_attn_cached(q, c, table, lens, out, ws, 1.0, 1, 32, w)
    for bad in (w[:3], w.double(), w.cpu(), w.transpose(0, 1)):
        with pytest.raises(ValueError):
            mq.mq_attn_cached(q, c, table, lens, out, ws, 1.0, 1, 32, bad)
    for bad in (ws.cpu(), ws.int()):
        with pytest.raises(ValueError):
            mq.mq_attn_cached(q, c, table, lens, out, bad, 1.0, 1, 32, w)
    with pytest.raises(mq.MQError) as e:
        mq.mq_attn_cached(q, c, table, lens, out, ws[:-16], 1.0, 1, 32, w)
    assert e.value.status == mq.MQ_ERR_WORKSPACE
    with pytest.raises(mq.MQError):
        mq.mq_attn_prompt(k, k, k, k[:, :1], cu, 3, math.nan)
    with pytest.raises(mq.MQError):  # in place
        mq.mq_kv_evict(c, table, lens, w, table, lens, torch.empty(2, 2, 4, dtype=torch.int32, device="cuda"), 1)
    with pytest.raises(ValueError):
        mq.KVCache(c.k_codes[:, :, :8], c.v_codes, c.k_scales, c.v_scales)
    with pytest.raises(ValueError):
        mq.KVCache(c.k_codes, c.v_codes[:3], c.k_scales, c.v_scales)


def test_cache_values():
    """KVCache.values decodes what mq_kv_append stored."""
    c = mq.KVCache.empty(2, 32, 1, 64)
    k = (torch.arange(64, device="cuda") - 32).bfloat16().expand(3, 1, 64).contiguous()
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    mq.mq_kv_append(k, -k / 32, c, table, zero, torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    kv, vv = c.values()
    near = torch.tensor(ref.e4m3_nearest(torch.arange(64).double() - 32).tolist()).float()
    assert torch.equal(kv[1, 0, :3].cpu(), near.expand(3, 64)) and not kv[1, 0, 3:16].any()
    assert torch.equal(vv[1, 0, :3].cpu(), -near.expand(3, 64) / 32)
