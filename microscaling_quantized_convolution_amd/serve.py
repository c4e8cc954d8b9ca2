"""One attention layer of a decoder that serves several sequences from an 8-bit cache.

``CachedAttention`` holds what such a layer keeps between calls, a paged key/value cache with its
page table, the sequences' lengths and the attention each cached token has received, and makes
the library's calls in their order:

  prefill   mq_attn_prompt over the packed prompts, then mq_kv_append of their keys and values
  decode    mq_kv_append of the new tokens, then mq_attn_cached, which adds up the weights
  evict     mq_kv_evict into fresh pages; the old ones become free

A prompt's own attention adds no weights: an eviction ranks its tokens by what the tokens generated
since gave them, and equal weights (none, right after ``prefill``) by position, the lowest first.
Projections, rotary embeddings and the rest of the layer are the caller's. Pages are handed out on
the host, so only ``prefill``, the first token of a page and ``evict`` copy a table to the device;
after an eviction the heads of a sequence hold different tokens (``positions`` tells which).
Everything runs on the current stream.

``python -m microscaling_quantized_convolution_amd.serve`` runs a small batch through all three.
"""
from __future__ import annotations

import math
from typing import List, Optional, Sequence

import torch

from . import (KVCache, attn_cached_workspace, mq_attn_cached, mq_attn_prompt, mq_kv_append,
               mq_kv_evict)


class CachedAttention:
    """Attention of ``n_seqs`` sequences, q_heads query heads on kv_heads key/value heads of
    head_dim, over at most max_len cached tokens each."""

    def __init__(self, n_seqs: int, max_len: int, q_heads: int, kv_heads: int, head_dim: int,
                 page_size: int = 64, num_pages: Optional[int] = None,
                 scale: Optional[float] = None, device="cuda"):
        if q_heads % kv_heads:
            raise ValueError(f"{q_heads} query heads on {kv_heads} key/value heads")
        self.n, self.q_heads = n_seqs, q_heads
        self.width = -(-max_len // page_size)
        self.max_len = max_len
        # room for every sequence at its longest, and for one being cut into fresh pages
        num_pages = (n_seqs + 1) * self.width if num_pages is None else num_pages
        self.cache = KVCache.empty(num_pages, page_size, kv_heads, head_dim, device)
        self.weights = torch.zeros(self.cache.weights_shape, device=device)
        self.scale = 1.0 / math.sqrt(head_dim) if scale is None else scale
        self.free = list(range(num_pages - 1, -1, -1))
        self.pages: List[List[int]] = [[] for _ in range(n_seqs)]
        self.held = [0] * n_seqs
        self.table = torch.full((n_seqs, self.width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device=device)
        self.steps = torch.arange(n_seqs + 1, dtype=torch.int32, device=device)
        self.ws: Optional[torch.Tensor] = None
        self.ws_len = 0  # tokens of a sequence that it is enough for
        self.positions: Optional[torch.Tensor] = None  # of the last eviction

    def _take(self, count: int) -> List[int]:
        if count > len(self.free):
            raise RuntimeError(f"{count} pages wanted, {len(self.free)} free")
        fresh = [self.free.pop() for _ in range(count)]
        if fresh:  # the weights of the pages' last owners are gone
            self.weights.index_fill_(0, torch.tensor(fresh, device=self.weights.device), 0.0)
        return fresh

    def _reserve(self, new: Sequence[int]):
        """Pages for new[s] more tokens of each sequence (all of them, or none and an error)."""
        page = self.cache.page_size
        for s, count in enumerate(new):
            if self.held[s] + count > self.max_len:
                raise ValueError(f"sequence {s}: {self.held[s]} + {count} tokens, at most "
                                 f"{self.max_len}")
        want = [max(0, -(-(self.held[s] + count) // page) - len(self.pages[s]))
                for s, count in enumerate(new)]
        fresh = self._take(sum(want))
        if not fresh:
            return
        for s, count in enumerate(want):
            self.pages[s] += fresh[:count]
            fresh = fresh[count:]
        self._copy_table()

    def _copy_table(self):
        rows = [p + [-1] * (self.width - len(p)) for p in self.pages]
        self.table.copy_(torch.tensor(rows, dtype=torch.int32))

    def prefill(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                lengths: Sequence[int]) -> torch.Tensor:
        """Prompts of the given lengths (0: none) for sequences that hold nothing, packed one after
        another: q [tokens][q_heads][dim], k and v [tokens][kv_heads][dim]. Returns their
        attention."""
        tokens = (len(q), len(k), len(v))
        if len(lengths) != self.n or min(lengths, default=0) < 0 or tokens != (sum(lengths),) * 3:
            raise ValueError(f"lengths {list(lengths)} for {self.n} sequences and {tokens} rows of q, k and v")
        if any(held and new for held, new in zip(self.held, lengths)):
            raise ValueError("a prompt for a sequence that holds tokens")
        self._reserve(lengths)
        cu = torch.tensor([sum(lengths[:s]) for s in range(self.n + 1)], dtype=torch.int32,
                          device=q.device)
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        mq_attn_prompt(q, k, v, out, cu, max(lengths, default=0), self.scale)
        mq_kv_append(k, v, self.cache, self.table, self.lens, cu)
        self._grow(lengths)
        return out

    def _grow(self, new: Sequence[int]):
        self.held = [h + c for h, c in zip(self.held, new)]
        self.lens.copy_(torch.tensor(self.held, dtype=torch.int32))

    def decode(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> torch.Tensor:
        """One new token of every sequence: q [n_seqs][q_heads][dim], k and v
        [n_seqs][kv_heads][dim]. Returns its attention over the cache, itself included."""
        self._reserve([1] * self.n)
        longest = max(self.held) + 1  # not max_len: the call's grid and scratch go by it
        if longest > self.ws_len:
            self.ws_len = min(self.max_len, 1 << (longest - 1).bit_length())
            self.ws = attn_cached_workspace(self.n, self.q_heads, self.cache.kv_heads,
                                            self.cache.head_dim, 1, self.ws_len, True, q.device)
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        mq_kv_append(k, v, self.cache, self.table, self.lens, self.steps)
        self.lens += 1
        try:
            mq_attn_cached(q, self.cache, self.table, self.lens, out, self.ws, self.scale, 1,
                           longest, self.weights)
        except Exception:
            self.lens -= 1  # the tokens just written are not held: the step can be made again
            raise
        self.held = [h + 1 for h in self.held]
        return out

    def evict(self, keep: int, recent: int):
        """Cut every sequence to `keep` tokens a head: the `recent` last ones and those that
        received the most attention. Shorter sequences stay as they are. The new pages have to be
        free beside the old ones: as many sequences are cut at a time as there are pages for, and
        there must be enough for one."""
        if keep < 0 or recent < 0:
            raise ValueError(f"keep {keep}, recent {recent}: expected 0 or more")
        need = -(-keep // self.cache.page_size)
        cut = [s for s, h in enumerate(self.held) if h > keep]
        if cut and need > len(self.free):
            raise RuntimeError(f"{need} pages wanted, {len(self.free)} free")
        dev = self.table.device
        at = torch.arange(keep, dtype=torch.int32, device=dev)
        held = torch.tensor(self.held, dtype=torch.int32, device=dev)[:, None, None]
        positions = torch.where(at < held, at, -1).repeat(1, self.cache.kv_heads, 1)
        try:
            while cut:
                count = len(self.free) // need if need else len(cut)
                self._cut(cut[:count], keep, recent, need, positions)
                cut = cut[count:]
            self.positions = positions
        finally:
            self._copy_table()
            self.lens.copy_(torch.tensor(self.held, dtype=torch.int32))

    def _cut(self, seqs: List[int], keep: int, recent: int, need: int, positions: torch.Tensor):
        """Cut these sequences, all longer than keep, into `need` fresh pages each."""
        dev = self.table.device
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        width = max(len(self.pages[s]) for s in seqs)
        table = ints([self.pages[s] + [-1] * (width - len(self.pages[s])) for s in seqs])
        lens = ints([self.held[s] for s in seqs])
        new_lens, kept = torch.empty_like(lens), torch.empty_like(positions[:len(seqs)])
        fresh = self._take(need * len(seqs))
        try:
            mq_kv_evict(self.cache, table, lens, self.weights, ints(fresh).view(len(seqs), need),
                        new_lens, kept, recent)
        except Exception:
            self.free += fresh  # nothing was launched
            raise
        positions[torch.tensor(seqs, device=dev)] = kept
        for i, s in enumerate(seqs):
            self.free += self.pages[s]
            self.pages[s], self.held[s] = fresh[i * need:(i + 1) * need], keep


def main():
    n, q_heads, kv_heads, dim, lengths = 3, 8, 2, 64, [200, 37, 90]
    layer = CachedAttention(n, 512, q_heads, kv_heads, dim, page_size=32)
    new = lambda tokens, heads: torch.randn(tokens, heads, dim, device="cuda").bfloat16()
    total = sum(lengths)
    out = layer.prefill(new(total, q_heads), new(total, kv_heads), new(total, kv_heads), lengths)
    print("prefill", tuple(out.shape), "tokens held", layer.held)
    for _ in range(50):
        out = layer.decode(new(n, q_heads), new(n, kv_heads), new(n, kv_heads))
    print("decode ", tuple(out.shape), "tokens held", layer.held)
    layer.evict(64, 16)
    out = layer.decode(new(n, q_heads), new(n, kv_heads), new(n, kv_heads))
    print("evict  ", tuple(out.shape), "tokens held", layer.held, "pages free", len(layer.free))


if __name__ == "__main__":
    main()
