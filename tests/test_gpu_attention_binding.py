"""What the binding of the attention calls refuses before it makes them (tensors on the GPU)."""
import pytest
import torch

import microscaling_quantized_convolution_amd as mq

pytestmark = pytest.mark.gpu


def test_lengths_have_one_dimension():
    """lens and cu are read as one number a sequence, whatever lies behind the first of them."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    c = mq.KVCache.empty(8, 16, 2, 64)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, table, cu = torch.empty_like(x), i32(*range(4)).view(2, 2), i32(0, 1, 3)
    w, new_lens = torch.zeros(c.weights_shape, device="cuda"), i32(0, 0)
    kept = torch.empty(2, 2, 4, dtype=torch.int32, device="cuda")
    for lens in (i32(0, 0, 0, 0).view(2, 2), i32(0)[0]):
        for call in (lambda: mq.mq_kv_append(x, x, c, table, lens, cu),
                     lambda: mq.mq_attn_cached(x[:2], c, table, lens, out[:2], None, 1.0, 1, 32),
                     lambda: mq.mq_kv_evict(c, table, lens, w, i32(4, 5).view(2, 1), new_lens, kept, 1)):
            with pytest.raises(ValueError, match="lens"):
                call()
    for bad in (i32(0, 1, 3, 3).view(2, 2), i32(0)[0]):
        with pytest.raises(ValueError, match="cu"):
            mq.mq_attn_prompt(x, x, x, out, bad, 3, 1.0)
