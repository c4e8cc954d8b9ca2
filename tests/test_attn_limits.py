"""Limits of the attention calls that the host decides (no GPU here): sizes that the kernels cannot
count, and workspaces that serve smaller calls too."""
import random

import pytest

import microscaling_quantized_convolution_amd as mq
from test_attn_abi import S0, cache


def evict(keep, new_width, **more):
    return mq.lib().mq_kv_evict(cache(**more), 0x100, 0x200, 0x300, 0x400, 0x500, 0x600, 1, 4, new_width,
                                keep, 0, S0)


@pytest.mark.parametrize("keep", [(1 << 30) + 1, (1 << 31) - 1024, (1 << 31) - 1])
def test_evict_refuses_more_kept_tokens_than_positions(keep):
    """The kernels step through the kept tokens in 32 bits."""
    page = 4096
    assert evict(keep, -(-keep // page), page=page) == mq.MQ_ERR_UNSUPPORTED


def test_workspace_serves_smaller_calls():
    """What the largest call needs is enough for fewer sequences, fewer new tokens, a smaller
    max_len, and without weights."""
    rng = random.Random(1)
    need = mq.mq_attn_cached_workspace_bytes
    spread = lambda top: int(2 ** rng.uniform(0, top))
    for _ in range(20000):
        heads, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 7, 20]), rng.choice([64, 96, 128, 192, 256])
        n, q_len, max_len, weights = spread(8), spread(4), spread(14), rng.random() < 0.5
        if rng.random() < 0.5:  # around a unit for every compute unit, and lengths of some tiles
            n, max_len = max(1, 256 // heads + rng.randint(0, 2)), rng.choice([1024, 1025, 4096, 4097])
        less = (rng.randint(max(1, n - 3), n) if rng.random() < 0.5 else rng.randint(1, n),
                rng.randint(1, q_len), rng.randint(0, max_len), weights and rng.random() < 0.5)
        large = need(n, heads * group, heads, dim, q_len, max_len, weights)
        small = need(less[0], heads * group, heads, dim, less[1], less[2], less[3])
        assert small <= large, (heads, group, dim, n, q_len, max_len, weights, less)
