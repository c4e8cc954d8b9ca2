"""The attention operators around the 8-bit key/value cache, as cases to be measured.

Four operators belong together: a prompt's attention (``mq_attn_prompt``), the quantizing write of
its keys and values into a paged cache (``mq_kv_append``), the attention of a few new tokens over
that cache (``mq_attn_cached``, which can also add up the weight each cached token received), and
the eviction of the tokens that received least (``mq_kv_evict``).

The cache holds E4M3 codes with one power-of-two scale (a byte e, the value 2^(e - 127)) for each
block of 16 tokens and head. Keys lie as [page][head][slot][dim], values as
[page][head][block][dim][slot of the block], scales as [page][head][block].

``own`` false computes each operator in its plain form, elementary torch operations in 32 bits;
``own`` true makes the package's calls.
"""
import math
import random

import torch

own = False

BLOCK = 16        # tokens that share a scale
E_MIN = 10        # smallest scale byte: its smallest code step is still a normal fp32 number
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # one generated token for each of a few sequences: what every decoding step pays
        {"name": "append step n6 h8 d128 bf16", "op": "append", "dtype": "bf16", "n": 6, "new": 1,
         "ragged": 0, "held": 1500, "heads": 8, "dim": 128, "page": 64},
        # a batch of prompts of different lengths enters the cache behind a shared beginning
        {"name": "append chunk n12 h4 d64 f16", "op": "append", "dtype": "f16", "n": 12,
         "new": 1021, "ragged": 3, "held": 333, "heads": 4, "dim": 64, "page": 32},
        # long prompts enter an empty cache
        {"name": "append prompts n4 h8 d128 bf16", "op": "append", "dtype": "bf16", "n": 4,
         "new": 16384, "ragged": 0, "held": 0, "heads": 8, "dim": 128, "page": 64},
        # one short conversation: latency alone counts
        {"name": "cached n1 len300 h8/2 d64 bf16", "op": "cached", "dtype": "bf16", "n": 1,
         "len": 300, "ragged": 0, "q_len": 1, "q_heads": 8, "heads": 2, "dim": 64, "page": 16,
         "weights": False},
        # a serving batch of mixed lengths
        {"name": "cached n32 len4096 h32/8 d128 bf16", "op": "cached", "dtype": "bf16", "n": 32,
         "len": 4096, "ragged": 5, "q_len": 1, "q_heads": 32, "heads": 8, "dim": 128, "page": 64,
         "weights": False},
        # one very long document: few rows, so the work is split along the cache
        {"name": "cached n1 len131071 h32/8 d128 f16", "op": "cached", "dtype": "f16", "n": 1,
         "len": 131071, "ragged": 0, "q_len": 1, "q_heads": 32, "heads": 8, "dim": 128,
         "page": 64, "weights": False},
        # four drafted tokens checked at once, the weights collected for a later eviction
        {"name": "cached n8 len8190 h16/4 q4 bf16 weights", "op": "cached", "dtype": "bf16",
         "n": 8, "len": 8190, "ragged": 7, "q_len": 4, "q_heads": 16, "heads": 4, "dim": 128,
         "page": 32, "weights": True},
        # one short question
        {"name": "prompt n1 len37 h8/2 d64 f16", "op": "prompt", "dtype": "f16", "n": 1,
         "len": 37, "ragged": 0, "q_heads": 8, "heads": 2, "dim": 64},
        # a packed batch of prompts of different lengths
        {"name": "prompt n8 len2047 h32/8 d128 bf16", "op": "prompt", "dtype": "bf16", "n": 8,
         "len": 2047, "ragged": 11, "q_heads": 32, "heads": 8, "dim": 128},
        # two long documents
        {"name": "prompt n2 len8192 h32/8 d128 bf16", "op": "prompt", "dtype": "bf16", "n": 2,
         "len": 8192, "ragged": 0, "q_heads": 32, "heads": 8, "dim": 128},
        # a few sequences cut back to a small budget
        {"name": "evict n2 len1000 h4 d64 keep256", "op": "evict", "n": 2, "len": 1000,
         "ragged": 0, "heads": 4, "dim": 64, "page": 16, "keep": 256, "recent": 32,
         "ties": False},
        # a batch of long contexts cut to a quarter
        {"name": "evict n8 len32768 h8 d128 keep8192", "op": "evict", "n": 8, "len": 32768,
         "ragged": 13, "heads": 8, "dim": 128, "page": 64, "keep": 8192, "recent": 512,
         "ties": False},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "cached", "prompt", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    heads = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 96, 128, 128, 256])
    page = rng.choice([16, 32, 48, 64, 128])
    n = _spread(rng, 1, 32)
    ragged = rng.randrange(1, 1 << 16)
    if op == "append":
        new = rng.choice([1, _spread(rng, 1, max(1, 65536 * 128 // (n * dim)) // 2)])
        return {"op": op, "dtype": dtype, "n": n, "new": new, "ragged": ragged,
                "held": rng.choice([0, _spread(rng, 1, 4000)]), "heads": heads, "dim": dim,
                "page": page}
    if op == "cached":
        q_len = rng.choice([1, 1, 1, 2, 5])
        return {"op": op, "dtype": dtype, "n": n,
                "len": _spread(rng, 1, 65536 * 128 // (n * dim) * 8 // (heads * q_len)),
                "ragged": ragged, "q_len": q_len, "q_heads": heads * rng.choice([1, 2, 4, 7, 8]),
                "heads": heads, "dim": dim, "page": page, "weights": rng.random() < 0.3}
    if op == "prompt":
        return {"op": op, "dtype": dtype, "n": n, "len": _spread(rng, 1, int(8192 / math.sqrt(n))),
                "ragged": ragged, "q_heads": heads * rng.choice([1, 2, 3, 4]), "heads": heads,
                "dim": min(dim, 128)}
    length = _spread(rng, 16, 262144 // n)
    keep = _spread(rng, 1, length)
    return {"op": op, "n": n, "len": length, "ragged": ragged, "heads": heads,
            "dim": min(dim, 128), "page": page, "keep": keep, "recent": rng.randint(0, keep),
            "ties": rng.random() < 0.3}


def _lengths(n, top, ragged):
    """Lengths of n sequences: all `top`, or (ragged) from `top` / 16 up to it, the longest first."""
    if not ragged:
        return [top] * n
    rng = random.Random(ragged)
    return [top] + [_spread(rng, max(1, top // 16), top) for _ in range(n - 1)]


def _counts(case):
    """(tokens held before, new tokens) of each sequence of an append."""
    new = _lengths(case["n"], case["new"], case["ragged"])
    rng = random.Random(case["ragged"] + 1)
    held = [case["held"] and max(0, case["held"] - rng.randrange(min(40, case["held"] + 1)))
            for _ in new]
    return held, new


def _ceil(a, b):
    return -(-a // b)


# ---- inputs ----------------------------------------------------------------------------------

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _gen(seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=_device(), dtype=dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=_device())


def _scale_bytes(amax):
    """Scale bytes of blocks with the largest magnitudes `amax` (fp32): the smallest power of two
    that brings them to 448 = 1.75 * 2^8 or less."""
    bits = amax.contiguous().view(torch.int32)
    e = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    return torch.where((bits >> 23) == 255, torch.full_like(e, 255), e.clamp(min=E_MIN))


def _power(e):
    """2^e of whole numbers e, exact."""
    return torch.ldexp(torch.ones((), device=e.device), e)


def _encode(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _filled_cache(g, pages, heads, page, dim):
    """Codes and scales of a cache full of normally distributed keys and values, whose size
    varies from block to block; a few of the keys' dimensions are far larger than the others."""
    out = []
    for value in (False, True):
        codes = torch.empty(pages, heads, page // BLOCK, BLOCK, dim, dtype=torch.uint8,
                            device=_device())
        scales = torch.empty(pages, heads, page // BLOCK, dtype=torch.uint8, device=_device())
        step = max(1, (1 << 26) // (heads * page * dim))
        for at in range(0, pages, step):
            x = _randn(g, min(step, pages - at), heads, page // BLOCK, BLOCK, dim)
            x *= torch.exp(0.5 * _randn(g, *x.shape[:3], 1, 1))
            if not value:
                x[..., ::37] *= 4.0
            e = _scale_bytes(x.abs().amax((3, 4)))
            codes[at:at + step] = _encode(x * _power(127 - e)[..., None, None])
            scales[at:at + step] = e.to(torch.uint8)
        codes = codes.transpose(3, 4).contiguous() if value else codes.view(pages, heads, page, dim)
        out += [codes, scales]
    return {"k_codes": out[0], "k_scales": out[1], "v_codes": out[2], "v_scales": out[3]}


def _table(g, pages, n, width, offset=0):
    """A page table of n rows: distinct pages of the pool in no order."""
    order = torch.randperm(pages, generator=g, device=_device()).to(torch.int32)
    return order[offset:offset + n * width].view(n, width).contiguous()


def _split_heads(g, tokens, q_heads, heads, dim, dtype):
    """Queries, keys and values as a projection leaves them: views of one [tokens][heads][dim]."""
    qkv = _randn(g, tokens, q_heads + 2 * heads, dim)
    qkv[:, q_heads:q_heads + heads, ::37] *= 3.0
    qkv = qkv.to(dtype)
    return qkv.split([q_heads, heads, heads], 1)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "append":
        held, new = _counts(case)
        width = max(_ceil(h + c, case["page"]) for h, c in zip(held, new))
        pages = case["n"] * width
        s["cache"] = _filled_cache(g, pages, case["heads"], case["page"], case["dim"])
        s["table"] = _table(g, pages, case["n"], width)
        _, s["k"], s["v"] = _split_heads(g, sum(new), case["heads"], case["heads"], case["dim"],
                                         DTYPES[case["dtype"]])
        s["held"], s["lens"], s["new"] = held, _ints(held), new
        s["cu"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
    elif op == "cached":
        lens = _lengths(case["n"], case["len"], case["ragged"])
        width = _ceil(max(lens), case["page"])
        pages = case["n"] * width
        s["cache"] = _filled_cache(g, pages, case["heads"], case["page"], case["dim"])
        s["table"] = _table(g, pages, case["n"], width)
        s["lens"], s["max_len"] = _ints(lens), max(lens)
        s["q"] = _randn(g, case["n"] * case["q_len"], case["q_heads"],
                        case["dim"]).to(DTYPES[case["dtype"]])
        s["out"] = torch.empty_like(s["q"])
        s["weights"] = (torch.rand(pages, case["heads"], case["page"], generator=g,
                                   device=_device()) if case["weights"] else None)
    elif op == "prompt":
        lens = _lengths(case["n"], case["len"], case["ragged"])
        s["cu"] = _ints([sum(lens[:i]) for i in range(len(lens) + 1)])
        s["max_len"] = max(lens)
        s["q"], s["k"], s["v"] = _split_heads(g, sum(lens), case["q_heads"], case["heads"],
                                              case["dim"], DTYPES[case["dtype"]])
        s["out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=s["q"].device)
    else:
        lens = _lengths(case["n"], case["len"], case["ragged"])
        width, to = _ceil(max(lens), case["page"]), _ceil(case["keep"], case["page"])
        pages = case["n"] * (width + to)
        s["cache"] = _filled_cache(g, pages, case["heads"], case["page"], case["dim"])
        table = _table(g, pages, 1, pages).view(-1)
        s["table"] = table[:case["n"] * width].view(case["n"], width).contiguous()
        s["new_table"] = table[case["n"] * width:].view(case["n"], to).contiguous()
        w = torch.rand(pages, case["heads"], case["page"], generator=g, device=_device())
        w = 0.01 / (w + 1e-3) - 0.0099  # most tokens receive little, a few very much
        s["weights"] = torch.floor(w * 256) / 256 if case["ties"] else w
        s["lens"] = _ints(lens)
        s["new_lens"] = torch.zeros_like(s["lens"])
        s["kept"] = torch.full((case["n"], case["heads"], case["keep"]), -1, dtype=torch.int32,
                               device=_device())
    return s


def _scale(dim):
    return 1.0 / math.sqrt(dim)


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _buffers(cache):
    """The cache as it is held: codes (as the E4M3 numbers that they are) and scale bytes."""
    return {"k": cache["k_codes"].view(torch.float8_e4m3fn), "k_scales": cache["k_scales"],
            "v": cache["v_codes"].view(torch.float8_e4m3fn), "v_scales": cache["v_scales"]}


def _handle(s):
    """The package's handle of the cache, which a program makes once."""
    if "handle" not in s:
        import microscaling_quantized_convolution_amd as mq
        c = s["cache"]
        s["handle"] = mq.KVCache(c["k_codes"], c["v_codes"], c["k_scales"], c["v_scales"])
    return s["handle"]


def _own_append(s):
    import microscaling_quantized_convolution_amd as mq
    mq.mq_kv_append(s["k"], s["v"], _handle(s), s["table"], s["lens"], s["cu"])
    return _buffers(s["cache"])


def _own_cached(s):
    import microscaling_quantized_convolution_amd as mq
    c = s["case"]
    if "ws" not in s:
        s["ws"] = mq.attn_cached_workspace(c["n"], c["q_heads"], c["heads"], c["dim"], c["q_len"],
                                           s["max_len"], s["weights"] is not None,
                                           s["q"].device)
    mq.mq_attn_cached(s["q"], _handle(s), s["table"], s["lens"], s["out"], s["ws"],
                      _scale(c["dim"]), c["q_len"], s["max_len"], s["weights"])
    return {"out": s["out"]} if s["weights"] is None else {"out": s["out"], "weights": s["weights"]}


def _own_prompt(s):
    import microscaling_quantized_convolution_amd as mq
    mq.mq_attn_prompt(s["q"], s["k"], s["v"], s["out"], s["cu"], s["max_len"],
                      _scale(s["case"]["dim"]))
    return {"out": s["out"]}


def _own_evict(s):
    import microscaling_quantized_convolution_amd as mq
    mq.mq_kv_evict(_handle(s), s["table"], s["lens"], s["weights"], s["new_table"],
                   s["new_lens"], s["kept"], s["case"]["recent"])
    return dict(_buffers(s["cache"]), weights=s["weights"], kept=s["kept"],
                new_lens=s["new_lens"])


# The plain forms. Held against exact(), which is written apart from them.

def _blocks(codes, value):
    """[pages][heads][blocks][16][dim] view of a cache's codes."""
    if value:
        return codes.transpose(3, 4)
    p, h, page, d = codes.shape
    return codes.view(p, h, page // BLOCK, BLOCK, d)


def _write_blocks(codes, scales, x, fresh, held, page, sub, value):
    """Fold x [blocks][16][heads][dim], where `fresh` [blocks][16], into the cache's blocks
    (page, sub), whose slots `held` already count; the blocks' other slots become zero."""
    view = _blocks(codes, value)
    x = torch.where(fresh[:, :, None, None], x, torch.zeros_like(x))
    e_new = _scale_bytes(x.abs().amax((1, 3)))
    e_old = scales[page, :, sub].int()
    e = torch.where(held.any(1)[:, None], torch.maximum(e_old, e_new), e_new)
    bad = (e == 255)[:, :, None, None]
    old = _decode(view[page, :, sub]) * _power(e_old - e)[:, :, None, None]
    both = torch.where(held[:, None, :, None], old,
                       x.transpose(1, 2) * _power(127 - e)[:, :, None, None])
    both = torch.where(bad | ~(held | fresh)[:, None, :, None], torch.zeros_like(both), both)
    view[page, :, sub] = _encode(both)
    scales[page, :, sub] = e.to(torch.uint8)


def _plain_append(s):
    c, cache, lens, cu = s["case"], s["cache"], s["lens"], s["cu"]
    per = [(h + n - 1) // BLOCK - h // BLOCK + 1 if n else 0 for h, n in zip(s["held"], s["new"])]
    total = sum(per)
    count = cu[1:] - cu[:-1]
    blocks = torch.where(count > 0, (lens + count - 1) // BLOCK - lens // BLOCK + 1, 0)
    first = torch.cumsum(blocks, 0) - blocks
    seq = torch.repeat_interleave(torch.arange(c["n"], device=lens.device), blocks,
                                  output_size=total)
    block = lens[seq] // BLOCK + torch.arange(total, device=lens.device) - first[seq]
    pos = block[:, None] * BLOCK + torch.arange(BLOCK, device=lens.device)
    held = pos < lens[seq][:, None]
    j = pos - lens[seq][:, None]
    fresh = (j >= 0) & (j < count[seq][:, None])
    rows = (cu[seq][:, None] + j).clamp(0, s["k"].shape[0] - 1).long()
    page = s["table"][seq, block // (c["page"] // BLOCK)].long()
    sub = block % (c["page"] // BLOCK)
    _write_blocks(cache["k_codes"], cache["k_scales"], s["k"][rows].float(), fresh, held, page,
                  sub, False)
    _write_blocks(cache["v_codes"], cache["v_scales"], s["v"][rows].float(), fresh, held, page,
                  sub, True)
    return _buffers(cache)


def _gather(codes, scales, table, value):
    """Keys or values [n][heads][slots][dim] in fp32, the pages of `table` one after another."""
    view, table = _blocks(codes, value), table.long()
    x = _decode(view[table]) * _power(scales[table].int() - 127)[..., None, None]
    n, width, heads, blocks, _, dim = x.shape
    return x.transpose(1, 2).reshape(n, heads, width * blocks * BLOCK, dim)


def _plain_cached(s):
    c, cache = s["case"], s["cache"]
    n, ql, hq, h, d = c["n"], c["q_len"], c["q_heads"], c["heads"], c["dim"]
    k = _gather(cache["k_codes"], cache["k_scales"], s["table"], False)
    v = _gather(cache["v_codes"], cache["v_scales"], s["table"], True)
    slots = k.shape[2]
    # rows of one key/value head: its query heads, then the new tokens
    q = s["q"].float().view(n, ql, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(n, h, -1, d)
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()) * _scale(d)
    pos = torch.arange(slots, device=q.device)
    last = s["lens"][:, None] - ql + torch.arange(ql, device=q.device)
    see = (pos <= last[..., None]).repeat(1, hq // h, 1)[:, None]
    scores = scores.masked_fill(~see, -math.inf)
    top = scores.amax(3, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(3, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = torch.matmul(p, v).view(n, h, hq // h, ql, d).permute(0, 3, 1, 2, 4)
    s["out"].copy_(out.reshape(n * ql, hq, d))
    if s["weights"] is None:
        return {"out": s["out"]}
    page = s["table"].long()[:, pos // c["page"]]
    slot = (pos % c["page"]).expand_as(page)
    s["weights"][page, :, slot] += p.sum(2).transpose(1, 2)
    return {"out": s["out"], "weights": s["weights"]}


def _plain_prompt(s):
    c, cu = s["case"], s["cu"]
    hq, h, d, top = c["q_heads"], c["heads"], c["dim"], s["max_len"]
    count = cu[1:] - cu[:-1]
    pos = torch.arange(top, device=cu.device)
    rows = (cu[:-1, None] + pos).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"][rows].float().transpose(1, 2)
    k = s["k"][rows].float().permute(0, 2, 3, 1).repeat_interleave(hq // h, 1).contiguous()
    v = s["v"][rows].float().transpose(1, 2).repeat_interleave(hq // h, 1).contiguous()
    scores = torch.matmul(q * _scale(d), k)
    scores.masked_fill_(pos[None, :] > pos[:, None], -math.inf)  # every row sees itself
    scores -= scores.amax(3, keepdim=True)
    scores.exp_()
    scores /= scores.sum(3, keepdim=True)
    out = torch.matmul(scores, v).transpose(1, 2)
    real = pos[None, :] < count[:, None]
    # rows of a shorter sequence's padding go to the last real row of it, and repeat its result
    at = torch.where(real, pos[None, :], count[:, None] - 1).long()
    out = torch.gather(out, 1, at[:, :, None, None].expand_as(out))
    s["out"][(cu[:-1, None] + at).long()] = out.to(s["out"].dtype)
    return {"out": s["out"]}


def _plain_evict(s):
    c, cache, weights, lens = s["case"], s["cache"], s["weights"], s["lens"]
    n, h, keep, recent, page = c["n"], c["heads"], c["keep"], c["recent"], c["page"]
    table, new_table = s["table"].long(), s["new_table"].long()
    w = weights[table].transpose(1, 2).reshape(n, h, -1)
    slots = w.shape[2]
    pos = torch.arange(slots, device=w.device)
    length = lens[:, None, None]
    w = torch.where(pos >= length - min(recent, keep), math.inf, w)
    w = torch.where(pos >= length, -math.inf, w)
    # equal weights keep their order, so that the lowest position wins
    order = torch.sort(w, dim=2, descending=True, stable=True).indices[:, :, :keep]
    order = torch.nn.functional.pad(order, (0, keep - order.shape[2]), value=slots)
    order = torch.where(torch.arange(keep, device=w.device) < length, order, slots)
    order = torch.sort(order, 2).values
    live = order < slots
    s["kept"].copy_(torch.where(live, order, -1))
    s["new_lens"].copy_(lens.clamp(max=keep))
    # whole blocks of the new pages, the slots past the kept tokens zero
    wide = _ceil(keep, BLOCK) * BLOCK
    order = torch.nn.functional.pad(torch.where(live, order, 0), (0, wide - keep))
    live = torch.nn.functional.pad(live, (0, wide - keep))
    seq = torch.arange(n, device=w.device)[:, None, None]
    head = torch.arange(h, device=w.device)[None, :, None]
    src = table[seq, order // page]
    at = order % page
    to = new_table[:, torch.arange(wide // BLOCK, device=w.device) // (page // BLOCK)]
    sub = (torch.arange(wide // BLOCK, device=w.device) % (page // BLOCK)).expand_as(to)
    used = (torch.arange(wide // BLOCK, device=w.device) * BLOCK
            < lens.clamp(max=keep)[:, None])[..., None]
    for_value = ((cache["k_codes"], cache["k_scales"], False),
                 (cache["v_codes"], cache["v_scales"], True))
    _move(*for_value[0], src, head, at, live, to, sub, used)
    _move(*for_value[1], src, head, at, live, to, sub, used)
    moved = torch.where(live, weights[src, head, at], 0.0)
    lane = torch.arange(wide, device=w.device)
    to, lane = new_table[:, lane // page], (lane % page).expand(n, -1)
    keepers = torch.where(used.repeat_interleave(BLOCK, 1),
                          moved.transpose(1, 2), weights[to, :, lane])
    weights[to, :, lane] = keepers
    return dict(_buffers(cache), weights=weights, kept=s["kept"], new_lens=s["new_lens"])


def _move(codes, scales, value, src, head, at, live, to, sub, used):
    """Copy the tokens (src, head, at) [n][heads][kept] into the blocks (to, sub) [n][blocks],
    each at the largest of its tokens' scales."""
    view = _blocks(codes, value)
    n, h, kept = src.shape
    x = _decode(view[src, head, at // BLOCK, at % BLOCK]).view(n, h, kept // BLOCK, BLOCK, -1)
    e_src = scales[src, head, at // BLOCK].int().view(n, h, kept // BLOCK, BLOCK)
    live = live.view(n, h, kept // BLOCK, BLOCK)
    e = torch.where(live, e_src, 0).amax(3)
    x = x * _power(e_src - e[..., None])[..., None]
    x = torch.where((live & (e != 255)[..., None])[..., None], x, torch.zeros_like(x))
    # blocks past the kept tokens stay as they are
    view[to, :, sub] = torch.where(used[..., None, None], _encode(x.transpose(1, 2)),
                                   view[to, :, sub])
    scales[to, :, sub] = torch.where(used, e.transpose(1, 2).to(torch.uint8), scales[to, :, sub])


_plain = {"append": _plain_append, "cached": _plain_cached, "prompt": _plain_prompt,
          "evict": _plain_evict}
_own = {"append": _own_append, "cached": _own_cached, "prompt": _own_prompt, "evict": _own_evict}


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    op, h, d = case["op"], case["heads"], case["dim"]
    if op == "append":
        tokens = sum(_counts(case)[1])
        return {"bytes": tokens * h * 2 * (3 * d + 1.0 / BLOCK), "flops": tokens * h * 2 * 3 * d}
    if op == "evict":
        lens = _lengths(case["n"], case["len"], case["ragged"])
        kept = sum(min(case["keep"], x) for x in lens)
        return {"bytes": sum(lens) * h * 4 + kept * h * (4 * (d + 1.0 / BLOCK) + 8),
                "flops": sum(lens) * h}
    lens = _lengths(case["n"], case["len"], case["ragged"])
    hq = case["q_heads"]
    if op == "cached":
        rows, seen = case["n"] * case["q_len"], sum(lens) * case["q_len"]
        per = 2 * (d + 1.0 / BLOCK) + (8 if case["weights"] else 0)
        return {"bytes": sum(lens) * h * per + rows * hq * d * 4, "flops": 4 * seen * hq * d}
    seen = sum(x * (x + 1) // 2 for x in lens)
    return {"bytes": sum(lens) * d * (4 * hq + 4 * h), "flops": 4 * seen * hq * d}


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "cached": _exact_cached, "prompt": _exact_prompt,
            "evict": _exact_evict}[case["op"]](s)


def _exact_values(cache):
    """The codes' numbers in 64 bits, and the scale bytes as whole numbers."""
    return {"k": cache["k_codes"].view(torch.float8_e4m3fn).double(),
            "v": cache["v_codes"].view(torch.float8_e4m3fn).double(),
            "k_scales": cache["k_scales"].long(), "v_scales": cache["v_scales"].long()}


def _nearest(x):
    """x rounded to the nearest E4M3 number (3 bits of fraction, exponents from -6), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_fold(x, e_was, was):
    """Codes' numbers and scale byte of a block [tokens][dim]: new rows x (64 bits) behind the held
    rows `was` (codes' numbers at the scale byte e_was)."""
    e = max(E_MIN, math.ceil(math.log2(max(float(x.abs().max()), 2.0 ** -140) / 448.0)) + 127)
    e = max(e, e_was)
    return torch.cat([_nearest(was * 2.0 ** (e_was - e)), _nearest(x * 2.0 ** (127 - e))]), e


def _exact_append(s):
    c, page = s["case"], s["case"]["page"]
    if sum(s["new"]) * c["heads"] > 60000:  # block by block: small cases alone take that long
        return None
    out = _exact_values(s["cache"])
    table, at = s["table"].tolist(), 0
    for i, (held, new) in enumerate(zip(s["held"], s["new"])):
        pos = held
        while pos < held + new:
            first = pos // BLOCK * BLOCK
            end = min(first + BLOCK, held + new)
            p, sub, was = table[i][pos // page], pos % page // BLOCK, pos - first
            for name, src in (("k", s["k"]), ("v", s["v"])):
                x = src[at:at + end - pos].double()
                for h in range(c["heads"]):
                    block = (out["k"][p, h, sub * BLOCK:(sub + 1) * BLOCK] if name == "k"
                             else out["v"][p, h, sub].t())
                    e_was = int(out[name + "_scales"][p, h, sub]) if was else 0
                    rows, e = _exact_fold(x[:, h], e_was, block[:was])
                    block[:end - first], block[end - first:] = rows, 0
                    out[name + "_scales"][p, h, sub] = e
            at += end - pos
            pos = end
    return out


def _exact_tokens(s, i, length, head):
    """Keys and values [length][dim] of one sequence and head, in 64 bits."""
    c, cache = s["case"], s["cache"]
    t = s["table"][i, :_ceil(length, c["page"])].long()
    k = cache["k_codes"][t, head].view(torch.float8_e4m3fn).double().reshape(-1, c["dim"])
    v = cache["v_codes"][t, head].view(torch.float8_e4m3fn).double()
    v = v.permute(0, 1, 3, 2).reshape(-1, c["dim"])
    ke = cache["k_scales"][t, head].double().reshape(-1).repeat_interleave(BLOCK)
    ve = cache["v_scales"][t, head].double().reshape(-1).repeat_interleave(BLOCK)
    return ((k * torch.exp2(ke - 127)[:, None])[:length],
            (v * torch.exp2(ve - 127)[:, None])[:length])


def _exact_cached(s):
    c = s["case"]
    group, ql = c["q_heads"] // c["heads"], c["q_len"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    weights = None if s["weights"] is None else s["weights"].double()
    for i, length in enumerate(s["lens"].tolist()):
        for head in range(c["heads"]):
            k, v = _exact_tokens(s, i, length, head)
            given = torch.zeros(length, dtype=torch.float64, device=k.device)
            for j in range(ql):
                see = length - ql + j + 1
                if see < 1:
                    continue
                q = s["q"][i * ql + j, head * group:(head + 1) * group].double()
                p = torch.softmax((q @ k[:see].t()) / math.sqrt(c["dim"]), 1)
                out[i * ql + j, head * group:(head + 1) * group] = p @ v[:see]
                given[:see] += p.sum(0)
            if weights is not None:
                pos = torch.arange(length, device=k.device)
                weights[s["table"][i].long()[pos // c["page"]], head, pos % c["page"]] += given
    return {"out": out} if weights is None else {"out": out, "weights": weights}


def _exact_prompt(s):
    c = s["case"]
    group = c["q_heads"] // c["heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    cu = s["cu"].tolist()
    for a, b in zip(cu, cu[1:]):
        tri = torch.ones(b - a, b - a, dtype=torch.bool, device=out.device).tril()
        for head in range(c["q_heads"]):
            q, k, v = (x.double() for x in (s["q"][a:b, head], s["k"][a:b, head // group],
                                            s["v"][a:b, head // group]))
            w = torch.where(tri, (q @ k.t()) / math.sqrt(c["dim"]), -math.inf)
            out[a:b, head] = torch.softmax(w, 1) @ v
    return {"out": out}


def _exact_evict(s):
    c, page, weights = s["case"], s["case"]["page"], s["weights"]
    if sum(s["lens"].tolist()) * c["heads"] > 100000:
        return None
    out = _exact_values(s["cache"])
    moved, kept = weights.double(), torch.full_like(s["kept"], -1)
    for i, length in enumerate(s["lens"].tolist()):
        t = s["table"][i].tolist()
        for h in range(c["heads"]):
            w = torch.cat([weights[p, h] for p in t])[:length].tolist()
            take = min(c["keep"], length)
            safe = min(c["recent"], take)
            best = sorted(range(length - safe), key=lambda j: (-w[j], j))[:take - safe]
            chosen = sorted(best) + list(range(length - safe, length))
            kept[i, h, :take] = torch.tensor(chosen, dtype=torch.int32)
            chosen = torch.tensor(chosen, device=weights.device)
            src, at = s["table"][i].long()[chosen // page], chosen % page
            for first in range(0, take, BLOCK):
                p, sub = int(s["new_table"][i, first // page]), first % page // BLOCK
                a, b = src[first:first + BLOCK], at[first:first + BLOCK]
                for name in ("k", "v"):
                    e = out[name + "_scales"][a, h, b // BLOCK]
                    x = (out["k"][a, h, b] if name == "k"
                         else out["v"][a, h, b // BLOCK, :, b % BLOCK])
                    block = (out["k"][p, h, sub * BLOCK:(sub + 1) * BLOCK] if name == "k"
                             else out["v"][p, h, sub].t())
                    block[:] = 0
                    block[:len(a)] = _nearest(x * torch.exp2((e - e.max()).double())[:, None])
                    out[name + "_scales"][p, h, sub] = e.max()
                moved[p, h, sub * BLOCK:(sub + 1) * BLOCK] = 0
                moved[p, h, sub * BLOCK:sub * BLOCK + len(a)] = weights[a, h, b].double()
    return dict(out, weights=moved, kept=kept, new_lens=s["lens"].clamp(max=c["keep"]))
