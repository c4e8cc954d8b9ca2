"""GPU tests of the attention calls where the numbers' range decides: probabilities many orders below
the largest against the definition in 64 bits, and rows without a finite result."""
import math

import pytest
import torch

import attn_reference as ref
import microscaling_quantized_convolution_amd as mq
from test_gpu_attention import filled, randn, run_cached

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- probabilities far below the largest -------------------------------------------------------

def prompt_bound(q, k, v, scale):
    """(out, bound) of one prompt of q [n][heads][dim] on one key/value head. On top of the bound
    for p rounded relative to itself, half precision has an absolute step: p is at least 2^-8 of its
    scale in the largest of each 64 tokens that a row sees, that scale is 2^11 and the smallest
    numbers are 2^-24 apart, so a token's p is off by 2^-25-11+8 = 2^-28 of that largest."""
    n, heads, dim = q.shape
    see = torch.ones(n, n, dtype=torch.bool).tril()
    kk, vv = k[:, 0].double(), v[:, 0].double()
    count = torch.arange(1, n + 1)[:, None]
    out = torch.zeros(q.shape, dtype=torch.float64)
    bound = torch.zeros_like(out)
    tiles = -(-n // 64)
    for h in range(heads):
        qq = q[:, h].double()
        p = torch.softmax(torch.where(see, qq @ kk.t() * scale, -math.inf), 1)
        out[:, h] = p @ vv
        size = torch.where(see, qq.abs() @ kk.abs().t() * abs(scale), 0.0).amax(1, keepdim=True)
        bound[:, h] = ref.attn_bound(out[:, h], p @ vv.abs(), ref.U[q.dtype],
                                     ref.score_error(dim, size), count, ref.U[q.dtype])
        if q.dtype == F16:
            for t in range(tiles):
                part = slice(64 * t, min(n, 64 * t + 64))
                top = torch.where(see[:, part], p[:, part], 0.0).amax(1, keepdim=True)
                bound[:, h] += 2.0 ** -28 * top * (see[:, part].double() @ vv[part].abs())
    return out, bound


def hold_prompt(logits, size, dim, dtype, seed):
    """A prompt whose token t has about logits[t] in every row and values of about size[t]."""
    gen = torch.Generator().manual_seed(seed)
    n = len(logits)
    q, k = (0.3 * torch.randn(n, h, dim, generator=gen) for h in (2, 1))
    q[..., 0], k[:, 0, 0] = 8.0, torch.tensor(logits, dtype=torch.float32)
    v = torch.randn(n, 1, dim, generator=gen).abs() * torch.tensor(size)[:, None, None]
    q, k, v = (x.to(dtype) for x in (q, k, v))
    want, bound = prompt_bound(q, k, v, 0.125)
    out = torch.full(q.shape, math.nan, dtype=dtype, device="cuda")
    mq.mq_attn_prompt(q.cuda(), k.cuda(), v.cuda(), out, ints([0, n]), n, 0.125)
    err = (out.cpu().double() - want).abs()
    worst = (err / bound).max().item()
    assert (err <= bound).all(), f"{worst} of the bound, {err.max()}"


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("above", [6.0, 14.0, 18.0, 22.0, 30.0])
@pytest.mark.parametrize("at", [0, 700])
def test_prompt_under_one_heavy_token(dtype, dim, above, at):
    """One token takes nearly all the weight but has no value: the result is what the others, `above`
    below it, give."""
    logits, size = [0.0] * 1500, [512.0] * 1500
    logits[at], size[at] = above, 0.0
    hold_prompt(logits, size, dim, dtype, int(above) + dim + at)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_prompt_steps_down_and_up(dtype):
    """Scores that fall by 9 and by 30 from 96 tokens to the next, and rise again, the values growing
    as the probabilities fall."""
    steps = [0, -9, -18, -27, -36, -6, -36, -20, -50, -10, 2, -7]
    logits = [float(s) for s in steps for _ in range(96)]
    size = [min(2.0 ** 12, math.exp(-0.25 * s)) for s in logits]  # 16 times that is a finite half
    hold_prompt(logits, size, 64, dtype, 5)


# ---- rows that are NaN -------------------------------------------------------------------------

@pytest.mark.parametrize("lens", [[70, 33], [70, 1500]])
def test_weights_of_tokens_that_a_nan_row_does_not_see(lens):
    """A row whose query holds a NaN gives NaN to the tokens that it sees and nothing to later ones."""
    q_len, page = 4, 16
    cache, table = filled(61, lens, page, 2, 64)
    q = randn(torch.Generator().manual_seed(31), 2 * q_len, 4, 64, dtype=BF16)
    got = []
    for rows in ((), ((0, 1), (q_len + 1, 2))):  # row 0 of sequence 0, row 1 of sequence 1
        for r, qh in rows:
            q[r, qh, 3] = math.nan
        w = torch.zeros(cache["k"].shape[:3], device="cuda")
        run_cached(cache, table, lens, q, q_len, 0.125, w)
        got.append(w.cpu())
    clean, bad = got
    for s, i, h in ((0, 0, 0), (1, 1, 1)):
        sees = lens[s] - q_len + i + 1
        at = [(table[s][t // page], t % page) for t in range(lens[s])]
        for t, (p, slot) in enumerate(at):
            assert math.isnan(bad[p, h, slot]) == (t < sees), t
            if t >= sees:
                assert bad[p, h, slot] == clean[p, h, slot] and clean[p, h, slot] > 0
            assert bad[p, 1 - h, slot] == clean[p, 1 - h, slot]


@pytest.mark.parametrize("n", [40, 1500])
def test_rows_whose_scores_are_all_minus_infinity(n):
    """The softmax of scores that are all -inf is NaN, as it is over a prompt; a row that sees no
    token stays 0, and so does what it gives."""
    cache, table = ref.empty_cache(2 + n // 16, 16, 1, 64), [list(range(2 + n // 16)), [-1] * (2 + n // 16)]
    k = torch.ones(n, 1, 64, dtype=BF16)
    ref.append(cache, k, k, table, [0, 0], [0, n, n])
    q = torch.zeros(2, 2, 64, dtype=BF16)
    q[:, 0, 5], q[:, 1, 5] = -math.inf, 1.0
    w = torch.zeros(cache["k"].shape[:3], device="cuda")
    out = run_cached(cache, table, [n, n], q, 1, 1.0)
    assert torch.isnan(out[0, 0]).all() and torch.equal(out[0, 1], torch.ones(64, dtype=BF16))
    assert not out[1].any()
    assert torch.equal(run_cached(cache, table, [n, n], q, 1, 1.0, w).nan_to_num(7.0), out.nan_to_num(7.0))
    row = w.cpu()[:, 0].flatten()
    assert torch.isnan(row[:n]).all() and not row[n:].any()
    whole = torch.empty(n, 2, 64, dtype=BF16, device="cuda")
    mq.mq_attn_prompt(q[:1].expand(n, 2, 64).contiguous().cuda(), k.cuda(), k.cuda(), whole, ints([0, n]), n, 1.0)
    assert torch.isnan(whole[:, 0]).all() and (whole[:, 1] == 1.0).all()


# ---- probabilities in more than 16 bits --------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens", [[300, 77], [2500, 1030]])
def test_cached_results_round_once(dtype, lens):
    """p goes into the second product to 2^-16 of itself, so that an output is off by its own
    rounding and little else, however much the values cancel."""
    dim, heads, group, scale = 64, 2, 3, 0.125
    cache, table = filled(71, lens, 32, heads, dim, dtype)
    q = randn(torch.Generator().manual_seed(41), len(lens), heads * group, dim, dtype=dtype)
    got = run_cached(cache, table, lens, q, 1, scale).double()
    for s, n in enumerate(lens):
        for h in range(heads):
            k, v = (ref.tokens(cache, side, table[s], n, h)[0] for side in ("k", "v"))
            rows = q[s, h * group:(h + 1) * group].double()
            p = torch.softmax(rows @ k.t() * scale, 1)
            size = (rows.abs() @ k.abs().t() * scale).amax(1, keepdim=True)
            want = p @ v
            bound = ref.attn_bound(want, p @ v.abs(), 2.0 ** -16, ref.score_error(dim, size), n, ref.U[dtype])
            err = (got[s, h * group:(h + 1) * group] - want).abs()
            assert (err <= bound).all(), f"{(err / bound).max()} of the bound"
