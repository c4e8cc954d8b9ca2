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
