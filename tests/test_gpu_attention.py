"""GPU tests of the key/value cache and attention calls against their 64-bit definitions
(attn_reference): the cache's bytes exactly, attention within the bounds derived there."""
import math
import random

import pytest
import torch

import attn_reference as ref
import microscaling_quantized_convolution_amd as mq

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
DIMS = [64, 96, 128, 192, 256]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def on_gpu(cache):
    return mq.KVCache(*(cache[n].cuda() for n in ("k", "v", "ks", "vs")))


def same_bytes(gpu, cache):
    for name, got in (("k", gpu.k_codes), ("v", gpu.v_codes), ("ks", gpu.k_scales), ("vs", gpu.v_scales)):
        got, want = got.cpu(), cache[name]
        if name in ("k", "v"):  # +0 and -0 are the same value
            got, want = torch.where(got == 0x80, 0, got), torch.where(want == 0x80, 0, want)
        assert torch.equal(got, want), name


def make_table(rng, lens, page, spare=2, extra=1):
    """Distinct pages in no order, `extra` unused entries a row that name no page."""
    width = max(1, max(-(-n // page) for n in lens)) + extra
    need = [-(-n // page) for n in lens]
    order = list(range(sum(need) + spare))
    rng.shuffle(order)
    rows = []
    for n in need:
        rows.append([order.pop() for _ in range(n)] + [-1, 1 << 30][:1] * (width - n))
    return rows, sum(need) + spare


def randn(gen, *shape, dtype):
    return torch.randn(shape, generator=gen).to(dtype)


def filled(seed, lens, page, heads, dim, dtype=BF16):
    """A cache on the CPU that holds lens[s] tokens of each sequence (stale bytes elsewhere)."""
    gen, rng = torch.Generator().manual_seed(seed), random.Random(seed)
    table, pages = make_table(rng, lens, page)
    cache = ref.empty_cache(pages, page, heads, dim)
    total = sum(lens)
    k, v = (randn(gen, total, heads, dim, dtype=dtype) for _ in range(2))
    size = torch.exp(torch.randn(total, 1, 1, generator=gen))
    k, v = (k * size).to(dtype), (v * size).to(dtype)
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    ref.append(cache, k, v, table, [0] * len(lens), cu)
    return cache, table


# ---- append ------------------------------------------------------------------------------------

@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_append_blocks(dim, dtype):
    """Blocks begun, continued, filled and left, scales that grow and do not, no new tokens."""
    rng, gen = random.Random(dim), torch.Generator().manual_seed(dim)
    page, heads = 48, 3
    held = [0, 1, 15, 16, 17, 47, 48, 0, 95, 30]
    new = [1, 14, 1, 16, 49, 1, 33, 0, 2, 100]
    lens = [a + b for a, b in zip(held, new)]
    table, pages = make_table(rng, lens, page)
    cache = ref.empty_cache(pages, page, heads, dim)
    for counts, at in ((held, [0] * len(held)), (new, held)):
        total = sum(counts)
        size = torch.exp(1.5 * torch.randn(total, 1, 1, generator=gen))
        k, v = ((torch.randn(total, heads, dim, generator=gen) * size).to(dtype) for _ in range(2))
        cu = [sum(counts[:i]) for i in range(len(counts) + 1)]
        g = on_gpu(cache)
        for _ in range(2):  # the second call changes nothing
            mq.mq_kv_append(k.cuda(), v.cuda(), g, ints(table), ints(at), ints(cu))
        ref.append(cache, k, v, table, at, cu)
        same_bytes(g, cache)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_append_extremes(dtype):
    """Largest and smallest magnitudes, ties of the rounding, zeros, NaN and infinities."""
    dim, page, heads = 64, 32, 1
    top = torch.finfo(dtype).max
    rows = torch.zeros(9 * 16, heads, dim)
    rows[0:16] = top
    rows[16:32] = torch.linspace(-top, top, 16 * dim).view(16, 1, dim)
    rows[32:48] = torch.arange(16 * dim).view(16, 1, dim) * (448.0 / (16 * dim))
    rows[48:64] = torch.finfo(dtype).tiny * torch.arange(16 * dim).view(16, 1, dim) / 64
    rows[80, 0, 3] = math.nan
    rows[96, 0, 63] = -math.inf
    rows[112:128] = 448.0
    rows[112, 0, 0] = 450.0
    rows[128:144] = 2.0 ** -20 * (1 + torch.arange(16 * dim).view(16, 1, dim) / 16)
    rows = rows.to(dtype)
    lens = [rows.shape[0]]
    table, pages = make_table(random.Random(0), lens, page)
    cache = ref.empty_cache(pages, page, heads, dim)
    g = on_gpu(cache)
    mq.mq_kv_append(rows.cuda(), -rows.cuda(), g, ints(table), ints([0]), ints([0, lens[0]]))
    ref.append(cache, rows, -rows, table, [0], [0, lens[0]])
    same_bytes(g, cache)
    # a poisoned block stays poisoned, a block begun anew does not
    g.k_scales.fill_(255)
    one = torch.ones(1, heads, dim, dtype=dtype, device="cuda")
    mq.mq_kv_append(one, one, g, ints(table), ints([3]), ints([0, 1]))
    mq.mq_kv_append(one, one, g, ints(table), ints([16]), ints([0, 1]))
    p = table[0][0]
    assert g.k_scales[p, 0, 0].item() == 255 and not g.k_codes[p, 0, :16].any()
    assert g.k_scales[p, 0, 1].item() == 127 - 8  # 1 <= 448 * 2^-8


def test_append_drops_what_has_no_place():
    """Tokens past the table's row, pages that do not exist, and a null tensor of no tokens."""
    dim, page, heads = 64, 16, 2
    gen = torch.Generator().manual_seed(3)
    table = [[0, -1, 2], [5, 1 << 30, 3]]
    cache = ref.empty_cache(6, page, heads, dim, fill=0x11)
    k, v = (randn(gen, 80, heads, dim, dtype=BF16) for _ in range(2))
    g = on_gpu(cache)
    args = (table, [0, 5], [0, 40, 80])
    mq.mq_kv_append(k.cuda(), v.cuda(), g, *(ints(a) for a in args))
    ref.append(cache, k, v, *args)
    same_bytes(g, cache)
    none = torch.empty(0, heads, dim, dtype=BF16, device="cuda")
    mq.mq_kv_append(none, none, g, ints(table), ints([0, 5]), ints([0, 0, 0]))
    same_bytes(g, cache)


def test_append_many_sequences():
    """More sequences than a wave searches at a time, most of them without new tokens."""
    dim, page, heads = 64, 16, 1
    rng, gen = random.Random(5), torch.Generator().manual_seed(5)
    new = [rng.choice([0, 0, 1, 3, 20]) for _ in range(300)]
    held = [rng.randrange(20) for _ in new]
    table, pages = make_table(rng, [a + b for a, b in zip(held, new)], page)
    cache = ref.empty_cache(pages, page, heads, dim, fill=0x22)
    k, v = (randn(gen, sum(new), heads, dim, dtype=BF16) for _ in range(2))
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    g = on_gpu(cache)
    mq.mq_kv_append(k.cuda(), v.cuda(), g, ints(table), ints(held), ints(cu))
    ref.append(cache, k, v, table, held, cu)
    same_bytes(g, cache)


# ---- attention over the cache ------------------------------------------------------------------

def run_cached(cache, table, lens, q, q_len, scale, weights=None, max_len=None, gpu=None, stream=None):
    g = gpu or on_gpu(cache)
    n, hq, d = len(lens), q.shape[1], q.shape[2]
    max_len = max(lens) if max_len is None else max_len
    heads = cache["k"].shape[1]
    ws = mq.attn_cached_workspace(n, hq, heads, d, q_len,
                                  max_len or len(table[0]) * cache["k"].shape[2], weights is not None)
    ws.fill_(0xFF)  # NaN in whatever is read before it is written
    out = torch.full(q.shape, math.nan, dtype=q.dtype, device="cuda")
    mq.mq_attn_cached(q.cuda(), g, ints(table), ints(lens), out, ws, scale, q_len, max_len, weights,
                      stream)
    return out.cpu()


def check_cached(cache, table, lens, q, q_len, scale, max_len=None):
    want, bound, given, given_bound = ref.cached(cache, q, table, lens, q_len, scale)
    first = torch.rand(cache["k"].shape[:3], generator=torch.Generator().manual_seed(1))
    w = first.cuda()
    for weights in (None, w):
        out = run_cached(cache, table, lens, q, q_len, scale, weights, max_len)
        err = (out.double() - want).abs()
        assert (err <= bound).all(), f"{err.max()} at bound {bound.flatten()[err.argmax()]}"
    err = (w.cpu().double() - first.double() - given).abs()
    assert (err <= given_bound + 2.0 ** -23 * (first + given)).all()


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_cached_lengths(dim, dtype):
    """Lengths from none and one to several tiles, pages that end inside a tile."""
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 130, 257]
    cache, table = filled(dim, lens, 48, 2, dim, dtype)
    q = randn(torch.Generator().manual_seed(dim), len(lens), 6, dim, dtype=dtype)
    check_cached(cache, table, lens, q, 1, 1 / math.sqrt(dim))


@pytest.mark.parametrize("heads,group,q_len", [(1, 1, 1), (1, 8, 1), (2, 7, 5), (3, 1, 17), (1, 16, 2),
                                               (2, 40, 1)])
def test_cached_rows(heads, group, q_len):
    """Row tiles that are part full, full and several; new tokens that see fewer tokens, or none."""
    lens = [3, 70, 1, 200]
    cache, table = filled(7, lens, 16, heads, 64)
    q = randn(torch.Generator().manual_seed(2), len(lens) * q_len, heads * group, 64, dtype=BF16)
    check_cached(cache, table, lens, q, q_len, 0.3)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_cached_split(dtype):
    """Sequences long enough to be split along the cache, next to short and empty ones."""
    lens = [3000, 0, 1, 1029]
    cache, table = filled(11, lens, 64, 1, 64, dtype)
    q = randn(torch.Generator().manual_seed(4), 2 * len(lens), 4, 64, dtype=dtype)
    check_cached(cache, table, lens, q, 2, 0.125)
    check_cached(cache, table, lens, q, 2, 0.125, max_len=0)  # the table's width


@pytest.mark.parametrize("n,heads", [(70, 1), (130, 2)])
def test_cached_many_ragged_sequences(n, heads):
    """More sequences than a wave has lanes, some of them empty: few heads, so that long sequences
    are cut along the cache, and enough for a workgroup to take a whole long sequence."""
    lens = [(37 * i) % 90 for i in range(n)]
    lens[3], lens[65], lens[n - 1] = 1500, 1100, 700
    cache, table = filled(37, lens, 32, heads, 64)
    q = randn(torch.Generator().manual_seed(14), n, 2 * heads, 64, dtype=BF16)
    check_cached(cache, table, lens, q, 1, 0.125)


def test_cached_sharp_and_signed_scales():
    """One token takes nearly all the weight; a negative and a zero scale."""
    lens = [100, 33]
    cache, table = filled(13, lens, 32, 2, 128)
    q = 6 * randn(torch.Generator().manual_seed(6), 2, 4, 128, dtype=BF16)
    for scale in (1.0, -0.5, 0.0):
        check_cached(cache, table, lens, q, 1, scale)


def test_cached_poison_reaches_only_those_who_see_it():
    """A block with the scale of NaN: rows that see it are NaN, rows before it and other heads are
    not, whichever side holds it."""
    lens, q_len = [40], 30  # rows see 11 ... 40 tokens: blocks 0, 1 and 2
    for side in ("ks", "vs"):
        cache, table = filled(17, lens, 16, 2, 64)
        q = randn(torch.Generator().manual_seed(8), q_len, 4, 64, dtype=BF16)
        clean = run_cached(cache, table, lens, q, q_len, 0.125)
        p = table[0][1]
        cache[side][p, 0, 0] = 255
        cache[side[0]][p, 0] = 0
        out = run_cached(cache, table, lens, q, q_len, 0.125)
        sees = torch.arange(11, 41) > 16
        assert torch.isnan(out[sees][:, :2]).all()
        assert torch.equal(out[~sees], clean[~sees]) and torch.equal(out[:, 2:], clean[:, 2:])
        assert torch.isfinite(clean).all()


def test_cached_skips_pages_that_do_not_exist():
    lens = [100, 90]
    cache, table = filled(19, lens, 16, 1, 64)
    table[0][2], table[1][0], table[1][5] = -1, 1 << 30, -7
    q = randn(torch.Generator().manual_seed(9), 2, 2, 64, dtype=BF16)
    check_cached(cache, table, lens, q, 1, 0.125)
    none = [[-1] * len(table[0])] * 2
    assert not run_cached(cache, none, lens, q, 1, 0.125).any()


def test_cached_lens_past_their_room():
    """Lengths beyond max_len or the table are read up to them, negative ones not at all."""
    lens = [64, 64, 64]
    cache, table = filled(23, lens, 32, 1, 64)
    table = [r[:2] for r in table]
    q = randn(torch.Generator().manual_seed(10), 3, 2, 64, dtype=BF16)
    got = run_cached(cache, table, [1000, -5, 64], q, 1, 0.125, max_len=64)
    want = run_cached(cache, table, [64, 0, 64], q, 1, 0.125, max_len=64)
    assert torch.equal(got, want) and not want[1].any()
    got = run_cached(cache, table, [64, 40, 64], q, 1, 0.125, max_len=40)
    want = run_cached(cache, table, [40, 40, 40], q, 1, 0.125, max_len=40)
    assert torch.equal(got, want)


def test_cached_strided_views():
    """q as part of a fused projection, out into a wider tensor."""
    lens, dim = [77, 5], 64
    cache, table = filled(29, lens, 16, 2, dim)
    fused = randn(torch.Generator().manual_seed(11), 2, 4 + 4, dim, dtype=BF16).cuda()
    wide = torch.full((2, 6, 2 * dim), 7.0, dtype=BF16, device="cuda")
    g = on_gpu(cache)
    ws = mq.attn_cached_workspace(2, 4, 2, dim, 1, 77)
    mq.mq_attn_cached(fused[:, 2:6], g, ints(table), ints(lens), wide[:, 1:5, dim:], ws, 0.125, 1, 77)
    want = run_cached(cache, table, lens, fused[:, 2:6].cpu(), 1, 0.125)
    assert torch.equal(wide[:, 1:5, dim:].cpu(), want)
    wide[:, 1:5, dim:] = 7.0
    assert (wide == 7.0).all()


def test_cached_repeats_and_streams():
    """The same bits on every call, on another stream too, and in a graph that is replayed."""
    lens = [2000, 700]
    cache, table = filled(31, lens, 64, 2, 64)
    gpu = on_gpu(cache)
    q = randn(torch.Generator().manual_seed(12), 2, 8, 64, dtype=BF16).cuda()
    shape = cache["k"].shape[:3]
    ws = mq.attn_cached_workspace(2, 8, 2, 64, 1, 2000, True)
    t, n = ints(table), ints(lens)
    outs = []

    def call(out, w, stream=None):
        mq.mq_attn_cached(q, gpu, t, n, out, ws, 0.125, 1, 2000, w, stream)

    side = torch.cuda.Stream()
    for stream in (None, None, side):
        out, w = torch.empty_like(q), torch.zeros(shape, device="cuda")
        torch.cuda.synchronize()
        call(out, w, stream)
        torch.cuda.synchronize()
        outs.append((out, w))
    for out, w in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(w, outs[0][1])
    out, w = torch.empty_like(q), torch.zeros(shape, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, w)
    for rep in range(3):
        w.zero_()
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, outs[0][0]) and torch.equal(w, outs[0][1]), rep


def test_offsets_past_32_bits():
    """A cache of over 4 GiB a side: pages at its end behave like those at its start."""
    dim, page, heads = 256, 1024, 8
    pages = (1 << 32) // (dim * page * heads) + 6
    lens = [1500, 1100]
    small = [[0, 1], [2, 3]]
    far = [[pages - 1, pages - 4], [pages - 2, pages - 3]]
    gen = torch.Generator().manual_seed(13)
    k, v = (randn(gen, sum(lens), heads, dim, dtype=BF16).cuda() for _ in range(2))
    q = randn(gen, 2, heads, dim, dtype=BF16).cuda()
    big = mq.KVCache.empty(pages, page, heads, dim)
    w = torch.zeros(big.weights_shape, device="cuda")
    ws = mq.attn_cached_workspace(2, heads, heads, dim, 1, 1500, True)
    outs, kept = [], []
    for table in (small, far):
        t, n = ints(table), ints(lens)
        mq.mq_kv_append(k, v, big, t, ints([0, 0]), ints([0, lens[0], sum(lens)]))
        out = torch.empty_like(q)
        mq.mq_attn_cached(q, big, t, n, out, ws, 0.0625, 1, 1500, w)
        outs.append(out)
        to = ints([[pages - 5], [pages - 6]] if table is far else [[4], [5]])
        nl, kp = torch.empty_like(n), torch.empty(2, heads, 300, dtype=torch.int32, device="cuda")
        mq.mq_kv_evict(big, t, n, w, to, nl, kp, 20)
        out = torch.empty_like(q)
        mq.mq_attn_cached(q, big, to, nl, out, ws, 0.0625, 1, 1500)
        outs.append(out)
        kept.append(kp)
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    assert torch.equal(kept[0], kept[1]) and torch.isfinite(outs[0]).all() and outs[0].any()


# ---- prompts -----------------------------------------------------------------------------------

def check_prompt(q, k, v, lens, scale, max_len=None):
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    want, bound = ref.prompt(q, k, v, cu, scale)
    out = torch.full(q.shape, math.nan, dtype=q.dtype, device="cuda")
    mq.mq_attn_prompt(q.cuda(), k.cuda(), v.cuda(), out, ints(cu), max_len or max(lens), scale)
    err = (out.cpu().double() - want).abs()
    assert (err <= bound).all(), f"{err.max()} at bound {bound.flatten()[err.argmax()]}"


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_prompt_lengths(dim, dtype):
    """Lengths from none and one across the tiles' edges, packed together."""
    gen = torch.Generator().manual_seed(dim)
    lens = [1, 0, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 0]
    q = randn(gen, sum(lens), 2, dim, dtype=dtype)
    k, v = (randn(gen, sum(lens), 1, dim, dtype=dtype) for _ in range(2))
    check_prompt(q, k, v, lens, 1 / math.sqrt(dim))


@pytest.mark.parametrize("heads,group,lens", [(2, 3, [300, 17]), (3, 1, [130, 260]), (1, 8, [200])])
def test_prompt_heads(heads, group, lens):
    gen = torch.Generator().manual_seed(heads)
    q = randn(gen, sum(lens), heads * group, 64, dtype=BF16)
    k, v = (randn(gen, sum(lens), heads, 64, dtype=BF16) for _ in range(2))
    check_prompt(q, k, v, lens, 0.2, max_len=1000)


def test_prompt_one_long_among_many_short():
    """Far more tiles in max_len than in the sequences, which are more than a wave searches at a
    time: the workgroups look for their tiles."""
    gen, rng = torch.Generator().manual_seed(26), random.Random(26)
    lens = [rng.choice([0, 1, 5, 40]) for _ in range(70)] + [390] + [rng.choice([0, 3]) for _ in range(30)]
    q = randn(gen, sum(lens), 2, 64, dtype=BF16)
    k, v = (randn(gen, sum(lens), 1, 64, dtype=BF16) for _ in range(2))
    for max_len in (390, 20000):
        check_prompt(q, k, v, lens, 0.125, max_len)


def test_prompt_sharp_and_signed_scales():
    gen = torch.Generator().manual_seed(21)
    lens = [150, 90]
    q = 5 * randn(gen, 240, 2, 64, dtype=F16)
    k, v = (randn(gen, 240, 1, 64, dtype=F16) for _ in range(2))
    for scale in (0.6, -0.6, 0.0):
        check_prompt(q, k, v, lens, scale)


def test_prompt_strided_views_and_max_len():
    """Parts of one fused projection; rows past max_len stay as they are."""
    gen = torch.Generator().manual_seed(22)
    lens, dim = [140, 60], 64
    fused = randn(gen, 200, 8, dim, dtype=BF16).cuda()
    q, k, v = fused.split([4, 2, 2], 1)
    out = torch.full((200, 4, dim), 7.0, dtype=BF16, device="cuda")
    cu = ints([0, 140, 200])
    mq.mq_attn_prompt(q, k, v, out, cu, 140, 0.125)
    dense = torch.empty_like(out)
    mq.mq_attn_prompt(q.contiguous(), k.contiguous(), v.contiguous(), dense, cu, 140, 0.125)
    assert torch.equal(out, dense)
    cut = torch.full_like(out, 7.0)
    mq.mq_attn_prompt(q, k, v, cut, cu, 100, 0.125)
    assert torch.equal(cut[:100], out[:100]) and (cut[100:140] == 7.0).all()
    assert torch.equal(cut[140:], out[140:])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["k", "v"])
def test_prompt_later_tokens_do_not_reach_earlier_rows(which, bad):
    """What a masked place holds adds nothing: rows before a NaN or an infinity keep their bits,
    rows that see it follow the formula."""
    gen = torch.Generator().manual_seed(23)
    n, at = 200, 75
    q = randn(gen, n, 2, 64, dtype=BF16).cuda()
    k, v = (randn(gen, n, 1, 64, dtype=BF16).cuda() for _ in range(2))
    cu, outs = ints([0, n]), []
    for poison in (False, True):
        if poison:
            (k if which == "k" else v)[at, 0, 5] = bad
        out = torch.empty_like(q)
        mq.mq_attn_prompt(q, k, v, out, cu, n, 0.125)
        outs.append(out)
    clean, got = outs
    assert torch.equal(got[:at], clean[:at]) and torch.isfinite(clean).all()
    if which == "v":
        assert not torch.isfinite(got[at:, :, 5]).any()
        other = [d for d in range(64) if d != 5]
        assert torch.equal(got[at:][..., other], clean[at:][..., other])
    elif bad != bad:
        assert torch.isnan(got[at:]).all()


def test_prompt_repeats_on_streams_and_in_a_graph():
    gen = torch.Generator().manual_seed(24)
    q = randn(gen, 500, 4, 128, dtype=BF16).cuda()
    k, v = (randn(gen, 500, 2, 128, dtype=BF16).cuda() for _ in range(2))
    cu = ints([0, 333, 500])
    want = torch.empty_like(q)
    mq.mq_attn_prompt(q, k, v, want, cu, 333, 0.1)
    torch.cuda.synchronize()
    side, out = torch.cuda.Stream(), torch.empty_like(q)
    torch.cuda.synchronize()
    mq.mq_attn_prompt(q, k, v, out, cu, 333, 0.1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mq.mq_attn_prompt(q, k, v, out, cu, 333, 0.1)
    for rep in range(3):
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep


# ---- evict -------------------------------------------------------------------------------------

def check_evict(seed, lens, page, heads, dim, keep, recent, weights=None, edit=None):
    cache, table = filled(seed, lens, page, heads, dim)
    rng = random.Random(seed + 1)
    to = -(-max(1, keep) // page)
    old = cache["k"].shape[0]
    new_pages = list(range(old, old + len(lens) * to))
    rng.shuffle(new_pages)
    new_table = [new_pages[i * to:(i + 1) * to] for i in range(len(lens))]
    more = ref.empty_cache(len(new_pages), page, heads, dim)
    cache = {n: torch.cat([cache[n], more[n]]) for n in cache}
    w = torch.rand(cache["k"].shape[:3], generator=torch.Generator().manual_seed(seed))
    if weights:
        w = weights(w)
    if edit:
        edit(cache, table, new_table)
    g, wg = on_gpu(cache), w.cuda()
    kept = torch.full((len(lens), heads, keep), -9, dtype=torch.int32, device="cuda")
    new_lens = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    mq.mq_kv_evict(g, ints(table), ints(lens), wg, ints(new_table), new_lens, kept, recent)
    want, want_lens = ref.evict(cache, w, table, lens, new_table, keep, recent)
    assert new_lens.tolist() == want_lens
    assert kept.tolist() == want
    same_bytes(g, cache)
    assert torch.equal(wg.cpu().nan_to_num(nan=-5.0), w.nan_to_num(nan=-5.0))


@pytest.mark.parametrize("dim", DIMS)
def test_evict_lengths(dim):
    check_evict(dim, [0, 1, 19, 20, 21, 100, 257], 48, 2, dim, 20, 5)


@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (16, 16), (17, 3), (33, 100), (300, 10), (0, 0)])
def test_evict_budgets(keep, recent):
    check_evict(41, [150, 33, 3], 16, 2, 64, keep, recent)


@pytest.mark.parametrize("kind", ["ties", "equal", "odd"])
def test_evict_order(kind):
    """Ties go to the lower position; NaN below everything, signed zeros equal, infinities at the
    ends."""
    def weights(w):
        if kind == "ties":
            return torch.floor(w * 4) / 4
        if kind == "equal":
            return torch.full_like(w, 0.5)
        special = torch.tensor([math.nan, 0.0, -0.0, math.inf, -math.inf, 1e-40, -1.0, 3.0])
        return special[(w * 8).long()]
    check_evict(43, [400, 129], 32, 2, 64, 100, 7, weights)


def test_evict_long():
    """More tokens than a workgroup has lanes, many times."""
    check_evict(47, [5000, 2311], 64, 1, 64, 700, 64, lambda w: torch.floor(w ** 8 * 4096) / 4096)


def test_evict_poison_and_missing_pages():
    def edit(cache, table, new_table):
        p = table[0][1]
        cache["ks"][p, 0, 0], cache["k"][p, 0] = 255, 0
        table[0][3] = -1
        table[1][0] = 1 << 29
        new_table[1][1] = -1
    check_evict(53, [100, 80], 16, 2, 64, 64, 10, edit=edit)
