"""GPU tests of attention weights where sequences read the same pages (a common beginning)."""
import math

import pytest
import torch

import attn_reference as ref
import microscaling_quantized_convolution_amd as mq
from test_gpu_attention import filled, ints, on_gpu, randn

pytestmark = pytest.mark.gpu


def check_weights(cache, table, lens, q, q_len, repeats=True):
    """Outputs and weights against the definition, which adds up what all sequences give a place;
    the sum of k sequences' shares and the weight that was there rounds k times."""
    n, hq, d = len(lens), q.shape[1], q.shape[2]
    want, bound, given, given_bound = ref.cached(cache, q, table, lens, q_len, 0.125)
    first = torch.rand(cache["k"].shape[:3], generator=torch.Generator().manual_seed(1))
    g = on_gpu(cache)
    ws = mq.attn_cached_workspace(n, hq, cache["k"].shape[1], d, q_len, max(lens), True)
    seen = []
    for _ in range(4):
        w, out = first.cuda(), torch.full(q.shape, math.nan, dtype=q.dtype, device="cuda")
        mq.mq_attn_cached(q.cuda(), g, ints(table), ints(lens), out, ws, 0.125, q_len, max(lens), w)
        assert ((out.cpu().double() - want).abs() <= bound).all()
        seen.append(w.cpu())
        err = (seen[-1].double() - first.double() - given).abs()
        slack = given_bound + (n + 1) * 2.0 ** -24 * (first + given)
        assert (err <= slack).all(), f"{err.max()} at {slack.flatten()[err.argmax()]}"
    if repeats:
        assert all(torch.equal(w, seen[0]) for w in seen)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [16, 32, 80])
def test_common_beginnings(dtype, page):
    """Two families with a beginning each, of different lengths; one sequence ends inside a common
    page, one is empty, one names the pages but holds no token of them."""
    lens = [400, 330, 0, 370, 90, 300, 280]
    cache, table = filled(page, lens, page, 2, 64, dtype)
    for s, of, pages in ((1, 0, 3), (3, 0, 4), (4, 0, 90 // page + 1), (2, 0, 2), (6, 5, 2)):
        table[s] = table[of][:pages] + table[s][pages:]
    q = randn(torch.Generator().manual_seed(3), 2 * len(lens), 4, 64, dtype=dtype)
    check_weights(cache, table, lens, q, 2)


def test_common_beginning_of_cut_sequences():
    lens = [2600, 1900, 2300]
    cache, table = filled(5, lens, 64, 1, 64)
    for s in (1, 2):
        table[s] = table[0][:20] + table[s][20:]
    q = randn(torch.Generator().manual_seed(4), len(lens), 2, 64, dtype=torch.bfloat16)
    check_weights(cache, table, lens, q, 1)


@pytest.mark.parametrize("longest", [150, 1300])
def test_common_beginning_of_many_sequences(longest):
    """More sequences than a wave has lanes, in one launch and cut along the cache."""
    lens = [70 + i % 5 for i in range(130)]
    lens[9], lens[100] = longest, longest - 3
    cache, table = filled(6, lens, 16, 1, 64)
    for s in range(2, 130, 3):
        table[s] = table[1][:4] + table[s][4:]
    table[100] = table[9][:6] + table[100][6:]
    q = randn(torch.Generator().manual_seed(5), len(lens), 2, 64, dtype=torch.bfloat16)
    check_weights(cache, table, lens, q, 1)


def test_a_page_at_two_places():
    """The same page at different places of two rows, and twice in one row: the sums are right."""
    lens = [96, 96, 64]
    cache, table = filled(7, lens, 16, 2, 64)
    table[1][4], table[1][1] = table[0][2], table[0][0]
    table[2][3] = table[2][0]
    q = randn(torch.Generator().manual_seed(6), len(lens), 4, 64, dtype=torch.bfloat16)
    check_weights(cache, table, lens, q, 1, repeats=False)
