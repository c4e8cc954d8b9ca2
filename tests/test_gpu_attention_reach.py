"""GPU tests of the attention calls' longer paths against the 64-bit definitions: sequences cut along
the cache in every dimension and in more than 64 pieces, candidates that do not fit on chip, NaN and
infinities in prompts of every dimension."""
import math
import random

import pytest
import torch

import attn_reference as ref
import microscaling_quantized_convolution_amd as mq
from test_gpu_attention import check_cached, check_evict, check_prompt, filled, ints, randn
from test_gpu_attention_range import prompt_bound

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
DIMS = [64, 96, 128, 192, 256]


# ---- attention over the cache ------------------------------------------------------------------

@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_cached_cut_and_joined(dim, dtype):
    """Pieces of two units of different lengths, next to sequences of one piece and of none."""
    lens = [1700, 0, 5, 1030]
    cache, table = filled(dim + 1, lens, 48, 2, dim, dtype)
    q = randn(torch.Generator().manual_seed(dim), 2 * len(lens), 6, dim, dtype=dtype)
    check_cached(cache, table, lens, q, 2, 1 / math.sqrt(dim))


def test_cached_more_pieces_than_lanes():
    """One unit of 67 pieces: maxima and sums of a row are found in several steps of a wave."""
    lens = [16900]
    cache, table = filled(3, lens, 64, 1, 64)
    q = randn(torch.Generator().manual_seed(3), 2, 2, 64, dtype=BF16)
    check_cached(cache, table, lens, q, 2, 0.125)


@pytest.mark.parametrize("unused", [-1, 1 << 30, -(1 << 31)])
def test_cached_unused_entries_name_no_page(unused):
    """Whatever the table holds behind a sequence's pages."""
    lens = [1100, 0, 17, 64]
    cache, table = filled(5, lens, 16, 2, 64)
    table = [[unused if p == -1 else p for p in row] for row in table]
    q = randn(torch.Generator().manual_seed(5), len(lens), 4, 64, dtype=BF16)
    check_cached(cache, table, lens, q, 1, 0.125)
    check_cached(cache, table, lens, q, 1, 0.125, max_len=0)


# ---- evict -------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["ties", "spread"])
@pytest.mark.parametrize("length,keep,recent", [(33500, 5000, 100), (40001, 39000, 0)])
def test_evict_more_candidates_than_fit_on_chip(kind, length, keep, recent):
    def weights(w):
        return torch.floor(w * 64) / 64 if kind == "ties" else w ** 8
    check_evict(length, [length, 300], 64, 1, 64, keep, recent, weights)


# ---- prompts -----------------------------------------------------------------------------------

@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_prompt_of_several_tiles(dim, dtype):
    gen = torch.Generator().manual_seed(dim)
    lens = [3, 411]
    q = randn(gen, sum(lens), 2, dim, dtype=dtype)
    k, v = (randn(gen, sum(lens), 1, dim, dtype=dtype) for _ in range(2))
    check_prompt(q, k, v, lens, 1 / math.sqrt(dim))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim,dtype", [(64, F16)] + [(d, t) for d in DIMS[1:] for t in (BF16, F16)])
def test_prompt_odd_values_reach_those_who_see_them(dim, dtype, bad):
    """Rows before a NaN or an infinity keep their bits, in every other dimension of the values all
    rows do; of the keys, rows follow the formula: a score of -inf takes the token out, anything else
    makes the row NaN."""
    gen = torch.Generator().manual_seed(dim)
    n, at, scale = 200, 75, 1 / math.sqrt(dim)
    q = randn(gen, n, 2, dim, dtype=dtype)
    k, v = (randn(gen, n, 1, dim, dtype=dtype) for _ in range(2))
    cu = ints([0, n])

    def run(k, v):
        out = torch.empty(q.shape, dtype=dtype, device="cuda")
        mq.mq_attn_prompt(q.cuda(), k.cuda(), v.cuda(), out, cu, n, scale)
        return out.cpu()
    clean = run(k, v)
    assert torch.isfinite(clean).all()
    odd = v.clone()
    odd[at, 0, 5] = bad
    got = run(k, odd)
    other = [d for d in range(dim) if d != 5]
    assert torch.equal(got[:at], clean[:at]) and torch.equal(got[..., other], clean[..., other])
    seen = got[at:, :, 5]
    assert torch.isnan(seen).all() if bad != bad else (seen == bad).all()
    odd = k.clone()
    odd[at, 0, 5] = bad
    got = run(odd, v)
    assert torch.equal(got[:at], clean[:at])
    out_of_it = q[at:, :, 5].float() * bad == -math.inf
    assert torch.equal(torch.isnan(got[at:]).all(2), ~out_of_it)
    # the token as it would be with the least weight that there is: none
    k0, v0 = (torch.cat([x[:at], x[at + 1:]]) for x in (k, v))
    want, bound = prompt_bound(torch.cat([q[:at], q[at + 1:]]), k0, v0, scale)
    rows = out_of_it[1:]  # behind the token itself
    err = (got[at + 1:].double() - want[at:]).abs()
    assert (err <= bound[at:])[rows].all()
