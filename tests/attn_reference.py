"""Plain 64-bit definitions of the attention and key/value cache calls, for the tests (CPU, torch
float64, one sequence and head at a time), and the error bounds the GPU results are held to.

A cache is a dict of CPU uint8 tensors k, v, ks, vs in the layouts of include/mq.h."""
import math

import torch

BLOCK, E_MIN = 16, 10
# largest relative error of one rounding to nearest
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def e4m3_nearest(x):
    """Nearest E4M3 value of |x| <= 448 in 64 bits: 3 bits of fraction down to the exponent -6."""
    exp = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(exp - 3)
    return torch.round(x / step) * step


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def codes_of(v):
    """Codes of exact E4M3 values."""
    return v.float().to(torch.float8_e4m3fn).view(torch.uint8)


def scale_byte(x):
    """Scale byte of a block with the elements x: search, not bit arithmetic."""
    if x.numel() == 0:
        return E_MIN
    top = x.abs().max().item()
    if not math.isfinite(top) or not torch.isfinite(x).all():
        return 255
    e = E_MIN
    while top > math.ldexp(448.0, e - 127):
        e += 1
    return e


def empty_cache(pages, page, heads, dim, fill=0x7F):
    """A cache of stale bytes (0x7F is E4M3's NaN)."""
    nb = page // BLOCK
    full = lambda *s: torch.full(s, fill, dtype=torch.uint8)
    return {"k": full(pages, heads, page, dim), "v": full(pages, heads, nb, dim, BLOCK),
            "ks": full(pages, heads, nb), "vs": full(pages, heads, nb)}


def _block(cache, side, p, h, b):
    """The codes of block b of a page and head as [16][dim] (a view)."""
    return cache["k"][p, h, b * BLOCK:(b + 1) * BLOCK] if side == "k" else cache["v"][p, h, b].t()


def append(cache, k, v, table, lens, cu):
    """In place. k, v [tokens][heads][dim]; table, lens, cu lists."""
    pages, heads, page, _ = cache["k"].shape
    for s, held in enumerate(lens):
        new = min(cu[s + 1] - cu[s], max(0, len(table[s]) * page - held))
        first = held // BLOCK * BLOCK if new > 0 else held  # no block is touched without a token
        while first < held + new:
            p, b = table[s][first // page], first % page // BLOCK
            lo, hi = max(0, held - first), min(BLOCK, held + new - first)
            row = cu[s] + first - held
            for side, src in (("k", k), ("v", v)):
                if not 0 <= p < pages:
                    continue
                for h in range(heads):
                    x = src[row + lo:row + hi, h].double()
                    block, was = _block(cache, side, p, h, b), int(cache[side + "s"][p, h, b])
                    e = max(scale_byte(x), was if lo else 0)
                    out = torch.zeros(block.shape, dtype=torch.float64)
                    if e != 255:
                        out[:lo] = e4m3_nearest(values(block[:lo]) * 2.0 ** (was - e))
                        out[lo:hi] = e4m3_nearest(x * 2.0 ** (127 - e))
                    block.copy_(codes_of(out))
                    cache[side + "s"][p, h, b] = e
            first += BLOCK


def tokens(cache, side, row, length, h):
    """(values [length][dim], which tokens exist) of one sequence and head; NaN where a scale is."""
    pages, _, page, dim = cache["k"].shape
    out, live = torch.zeros(length, dim, dtype=torch.float64), torch.zeros(length, dtype=torch.bool)
    for t in range(0, length, BLOCK):
        p, b, c = row[t // page], t % page // BLOCK, min(BLOCK, length - t)
        if 0 <= p < pages:
            e = int(cache[side + "s"][p, h, b])
            f = math.nan if e == 255 else 2.0 ** (e - 127)
            out[t:t + c], live[t:t + c] = values(_block(cache, side, p, h, b)[:c].contiguous()) * f, True
    return out, live


def _attend(q, k, v, see, scale):
    """One row: out, p, sum p|v|, sum |q k| * |scale| at its largest."""
    s = (k @ q) * scale
    s[~see] = -math.inf
    if not see.any():
        z = torch.zeros(v.shape[1], dtype=torch.float64)
        return z, torch.zeros(len(k), dtype=torch.float64), z, 0.0
    p = torch.softmax(s, 0)
    out, mass = p[see] @ v[see], p[see] @ v[see].abs()
    size = ((k[see].abs() @ q.abs()) * abs(scale)).max().item()
    return out, torch.where(see, p, 0.0), mass, size


def cached(cache, q, table, lens, q_len, scale):
    """(out, bound, weights added, their bound); q [n * q_len][q_heads][dim] of a 16-bit type."""
    _, heads, page, dim = cache["k"].shape
    hq = q.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64)
    bound = torch.zeros_like(out)
    given = torch.zeros(cache["k"].shape[:3], dtype=torch.float64)
    given_bound = torch.zeros_like(given)
    for s, length in enumerate(lens):
        length = min(length, len(table[s]) * page)
        for h in range(heads):
            k, live = tokens(cache, "k", table[s], length, h)
            v, _ = tokens(cache, "v", table[s], length, h)
            for i in range(q_len):
                see = live & (torch.arange(length) <= length - q_len + i)
                for qh in range(h * (hq // heads), (h + 1) * (hq // heads)):
                    r = s * q_len + i
                    o, p, mass, size = _attend(q[r, qh].double(), k, v, see, scale)
                    out[r, qh] = o
                    eps = score_error(dim, size)
                    # p in bf16, or (float16) in two bf16 parts
                    u = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -16
                    bound[r, qh] = attn_bound(o, mass, u, eps, length, U[q.dtype])
                    for t in torch.nonzero(see).flatten().tolist():
                        at = (table[s][t // page], h, t % page)
                        given[at] += p[t]
                        given_bound[at] += p[t] * (2 * eps + (length + 4) * 2.0 ** -24)
    return out, bound, given, given_bound


def score_error(dim, size):
    """Bound of a score's absolute error in fp32 (natural units): the products are exact, their sum
    of `dim` terms of total magnitude `size` rounds dim times, and the scaling, the subtraction of
    the maximum and 2^x round a few times more relative to |score| <= size."""
    return (dim + 8) * 2.0 ** -24 * size + 2.0 ** -22


def attn_bound(out, mass, u_p, eps, length, u_out):
    """|error| of an output: every p is off by eps in its exponent (so is the sum), by u_p from its
    rounding, the sum over `length` tokens rounds in fp32, and the result once to its type."""
    rel = u_p + 2 * eps + (length + 4) * 2.0 ** -24
    return rel * (1 + u_out) * mass + u_out * out.abs() + 2.0 ** -24


def prompt(q, k, v, cu, scale):
    """(out, bound) of causal attention; q, k, v [tokens][heads][dim] of a 16-bit type."""
    hq, heads, dim = q.shape[1], k.shape[1], q.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64)
    bound = torch.zeros_like(out)
    for a, b in zip(cu, cu[1:]):
        for qh in range(hq):
            h = qh // (hq // heads)
            kk, vv = k[a:b, h].double(), v[a:b, h].double()
            for i in range(b - a):
                see = torch.arange(b - a) <= i
                o, _, mass, size = _attend(q[a + i, qh].double(), kk, vv, see, scale)
                out[a + i, qh] = o
                bound[a + i, qh] = attn_bound(o, mass, U[q.dtype], score_error(dim, size), i + 1,
                                              U[q.dtype])
    return out, bound


def evict(cache, weights, table, lens, new_table, keep, recent):
    """In place. Returns (kept as lists, new lens)."""
    pages, heads, page, dim = cache["k"].shape
    source = {n: t.clone() for n, t in cache.items()}
    w_src = weights.clone()
    kept, new_lens = [], []
    for s, length in enumerate(lens):
        length = min(length, len(table[s]) * page)
        take = min(length, keep)
        safe = min(recent, take)
        new_lens.append(take)
        kept.append([])
        for h in range(heads):
            def weight(t):
                p = table[s][t // page]
                w = w_src[p, h, t % page].item() if 0 <= p < pages else math.nan
                return (0, 0.0) if math.isnan(w) else (1, w)
            others = sorted(range(length - safe), key=lambda t: (tuple(-c for c in weight(t)), t))
            chosen = sorted(others[:take - safe]) + list(range(length - safe, length))
            kept[s].append(chosen + [-1] * (keep - take))
            for first in range(0, take, BLOCK):
                part = chosen[first:first + BLOCK]
                p, b = new_table[s][first // page], first % page // BLOCK
                if not 0 <= p < pages:
                    continue
                for side in ("k", "v"):
                    x, es = torch.zeros(BLOCK, dim, dtype=torch.float64), []
                    for i, t in enumerate(part):
                        o = table[s][t // page]
                        if 0 <= o < pages:
                            x[i] = values(_block(source, side, o, h, t % page // BLOCK)[t % BLOCK].contiguous())
                            es.append(int(source[side + "s"][o, h, t % page // BLOCK]))
                        else:
                            es.append(E_MIN)
                    e = max(es)
                    y = torch.zeros_like(x)
                    if e != 255:
                        for i, ei in enumerate(es):
                            y[i] = e4m3_nearest(x[i] * 2.0 ** (ei - e))
                    _block(cache, side, p, h, b).copy_(codes_of(y))
                    cache[side + "s"][p, h, b] = e
                new = torch.zeros(BLOCK)
                for i, t in enumerate(part):
                    o = table[s][t // page]
                    if 0 <= o < pages:
                        new[i] = w_src[o, h, t % page]
                weights[p, h, b * BLOCK:(b + 1) * BLOCK] = new
    return kept, new_lens
