"""An attention layer over packed matrices: the q, k, v and o products with
rotary positions, the paged cache and the attention between them.

``AttentionLayer`` is the shortest complete use of wal_rope_freqs,
wal_kv_write, wal_attn_paged and wal_attn_prompt: forward() takes the new
tokens of any sequences, whole prompts, chunks of them and single tokens
alike.  examples/attention_layer.py runs one.

The products and the attention are libwal's (prompt() rounds v to bf16 with
torch); this module keeps the page lists.
"""
from __future__ import annotations

from operator import index
from typing import List, Sequence

import numpy as np

from . import (WAL_KV_BF16, WAL_MAX_BATCH, WAL_ROPE_HALF, make_kv_desc, make_rope_desc, wal_attn_paged,
               wal_attn_paged_workspace_size, wal_attn_prompt, wal_gemm_prefill, wal_gemm_small, wal_head_norm,
               wal_kv_size, wal_kv_write, wal_prefill_workspace_size, wal_rope, wal_rope_freqs, wal_workspace_size)


def _counts(new: Sequence[int], *rows) -> List[int]:
    """Counts of tokens, whose sum is every tensor's number of rows."""
    new = [index(n) for n in new]
    if not new or min(new) < 0:
        raise ValueError(f"counts of tokens {new}: at least one, none below 0")
    for t in rows:
        if t.shape[0] != sum(new):
            raise ValueError(f"{t.shape[0]} rows for {sum(new)} tokens")
    return new


def _sequences(seqs: Sequence[int], n: int, new=None) -> List[int]:
    """Distinct sequences of a layer with n, as many as there are counts of new tokens."""
    seqs = [index(s) for s in seqs]
    if new is not None and len(seqs) != len(new):
        raise ValueError(f"{len(seqs)} sequences with {len(new)} counts of new tokens")
    if len(set(seqs)) != len(seqs):
        raise ValueError(f"a sequence more than once in {seqs}")
    for s in seqs:
        if not 0 <= s < n:
            raise ValueError(f"sequence {s} of a layer with {n}")
    return seqs


class AttentionLayer:
    """q, k, v, o: (info, packed bytes on the GPU) of the layer's matrices; the
    heads' size is head_dim.  The cache holds n_pages pages of page_size
    tokens for max_seqs sequences.  q_norm, k_norm: weights [head_dim] of norms of the heads of q and
    of k before the rotation (one type, fp32 or bf16), with eps; None: there is none."""

    def __init__(self, q, k, v, o, head_dim: int, n_pages: int, max_seqs: int, page_size: int = 64,
                 fmt: int = WAL_KV_BF16, rope=None, layout: int = WAL_ROPE_HALF, q_norm=None, k_norm=None,
                 eps: float = 1e-6):
        import torch
        self.torch, self.dev = torch, q[1].device
        self.mats, self.head_dim, self.layout = (q, k, v, o), head_dim, layout
        self.q_norm, self.k_norm, self.eps = q_norm, k_norm, eps
        self.q_heads, self.kv_heads = q[0].d.out // head_dim, k[0].d.out // head_dim
        turns, self.magnitude = wal_rope_freqs(rope if rope is not None else make_rope_desc(head_dim, base=1e6))
        self.turns = torch.from_numpy(turns).to(self.dev)
        self.desc = make_kv_desc(n_pages, page_size, self.kv_heads, head_dim, fmt)
        self.cache = torch.empty(wal_kv_size(self.desc).total_bytes, dtype=torch.uint8, device=self.dev)
        self.free = list(range(n_pages))
        self.pages: List[List[int]] = [[] for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.ws = {}

    def _workspace(self, what: str, n: int):
        """A zeroed buffer for the products and one for the attention, each of which keeps its own first
        words zero between calls; grown when a call needs more."""
        if what not in self.ws or self.ws[what].numel() < n:
            self.ws[what] = self.torch.zeros(max(n, 16), dtype=self.torch.uint8, device=self.dev)
        return self.ws[what]

    def _product(self, m, X):
        info, W = m
        Y = self.torch.empty((X.shape[0], info.d.out), device=self.dev)
        if X.shape[0] <= WAL_MAX_BATCH:
            return wal_gemm_small(info, W, X, Y, ws=self._workspace("product", wal_workspace_size(info, X.shape[0])))
        return wal_gemm_prefill(info, W, X, Y, ws=self._workspace("prompt", wal_prefill_workspace_size(info, X.shape[0])))

    def _checked(self, seqs: Sequence[int], new: Sequence[int], *rows):
        """seqs and new as lists of int: distinct sequences of the layer with as many new tokens as each tensor has rows."""
        new = _counts(new, *rows)
        return _sequences(seqs, len(self.lens), new), new

    def _place(self, seqs: Sequence[int], new: Sequence[int]):
        """Where the new tokens go: their cache slots and positions, the sequences' pages with those that they
        need besides, and their lengths.  Nothing is changed yet."""
        size, slots, pos, pages, lens = self.desc.page_size, [], [], [], []
        left = len(self.free)
        for s, n in zip(seqs, new):
            t = np.arange(self.lens[s], self.lens[s] + n)
            more = max(-(-(self.lens[s] + n) // size) - len(self.pages[s]), 0)
            if more > left:
                raise RuntimeError(f"sequence {s} needs {more} more pages; the cache has {left} left")
            pages.append(self.pages[s] + self.free[left - more:left] if more else self.pages[s])
            left -= more
            slots.append(np.asarray(pages[-1], np.int64)[t // size] * size + t % size if n else t)
            pos.append(t)
            lens.append(self.lens[s] + n)
        return np.concatenate(slots).astype(np.int32), np.concatenate(pos).astype(np.int32), pages, lens

    def _keep(self, seqs: Sequence[int], pages: List[List[int]], lens: List[int]):
        """Counts the tokens of a call as kept in the cache, and their pages as taken."""
        del self.free[len(self.free) - sum(len(p) - len(self.pages[s]) for s, p in zip(seqs, pages)):]
        for s, p, n in zip(seqs, pages, lens):
            self.pages[s], self.lens[s] = p, n

    def release(self, s: int):
        s, = _sequences([s], len(self.lens))
        self.free += self.pages[s]
        self.pages[s], self.lens[s] = [], 0

    def attend(self, Q, K, V, seqs: Sequence[int], new: Sequence[int]):
        """The part between the products: Q, K, V (fp32 or bf16) of new[i] tokens of
        sequence seqs[i] each, one after another -> bf16 [n][q_heads * head_dim].  A call that raises, for want of
        pages (RuntimeError: release a sequence and call again) or otherwise, leaves the sequences as they were."""
        seqs, new = self._checked(seqs, new, Q, K, V)
        out, pages, lens = self._attend(Q, K, V, seqs, new)
        self._keep(seqs, pages, lens)
        return out

    def _attend(self, Q, K, V, seqs: Sequence[int], new: Sequence[int]):
        """attend() up to its launches, and the sequences' pages and lengths after it."""
        torch = self.torch
        slots, pos, pages, lens = self._place(seqs, new)
        tables = np.zeros((len(seqs), max(1, max(len(p) for p in pages))), np.int32)
        for i, p in enumerate(pages):
            tables[i, :len(p)] = p
        slots, pos, lens_dev, starts, tables = self._put(slots, pos, lens, np.cumsum([0] + new), tables)
        q, out = (torch.empty(Q.shape, dtype=torch.bfloat16, device=self.dev) for _ in range(2))
        wal_kv_write(self.desc, self.cache, slots, K, V, pos=pos, turns=self.turns, layout=self.layout,
                     magnitude=self.magnitude, Q=Q, Q_out=q, q_norm=self.q_norm, k_norm=self.k_norm, eps=self.eps)
        max_new, max_len = max(new), max(lens)
        ws = self._workspace("attention", wal_attn_paged_workspace_size(self.desc, self.q_heads, len(seqs),
                                                                        Q.shape[0], max_new, max_len))
        wal_attn_paged(self.desc, self.cache, tables, lens_dev, starts, q, out, ws, max_new=max_new, max_len=max_len)
        return out, pages, lens

    def _put(self, *arrays):
        """int32 arrays to the GPU in one copy."""
        arrays = [np.asarray(x, np.int32) for x in arrays]
        flat = self.torch.from_numpy(np.concatenate([x.ravel() for x in arrays])).to(self.dev)
        at = np.cumsum([0] + [x.size for x in arrays])
        return [flat[i:j].view(x.shape) for x, i, j in zip(arrays, at[:-1], at[1:])]

    def forward(self, X, seqs: Sequence[int], new: Sequence[int]):
        """X bf16 [n][hidden] -> fp32 [n][hidden], the new tokens of the sequences kept in the cache (of none of them,
        if the call raises)."""
        seqs, new = self._checked(seqs, new, X)
        Q, K, V = (self._product(m, X) for m in self.mats[:3])
        out, pages, lens = self._attend(Q, K, V, seqs, new)
        Y = self._product(self.mats[3], out)
        self._keep(seqs, pages, lens)
        return Y

    def prompt(self, X, lens: Sequence[int]):
        """The same for whole prompts that need no cache (scoring): X bf16, prompts one after another."""
        torch, lens = self.torch, _counts(lens, X)
        Q, K, V = (self._product(m, X) for m in self.mats[:3])
        pos = torch.from_numpy(np.concatenate([np.arange(n) for n in lens]).astype(np.int32)).to(self.dev)
        q, k = (torch.empty(t.shape, dtype=torch.bfloat16, device=self.dev) for t in (Q, K))
        for t, r, w in ((Q, q, self.q_norm), (K, k, self.k_norm)):
            if w is None:
                wal_rope(t, r, pos, self.turns, self.head_dim, layout=self.layout, magnitude=self.magnitude)
            else:
                wal_head_norm(t, r, w, self.head_dim, eps=self.eps, pos=pos, turns=self.turns, layout=self.layout,
                              magnitude=self.magnitude)
        starts = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device=self.dev)
        out = torch.empty_like(q)
        wal_attn_prompt(q, k, V.to(torch.bfloat16), starts, out, self.head_dim, max(lens))
        return self._product(self.mats[3], out)


def packed_layer(seed: int, hidden: int, q_heads: int, kv_heads: int, head_dim: int, rank: int = 16):
    """Random packed q, k, v, o of a layer, on the GPU."""
    import torch

    import synth

    from . import pack_matrix
    out = []
    for i, (rows, cols) in enumerate([(q_heads * head_dim, hidden)] + 2 * [(kv_heads * head_dim, hidden)]
                                     + [(hidden, q_heads * head_dim)]):
        blob, info = pack_matrix(synth.make_matrix(seed, i, rows, cols, k=8, n_paths=1, rank=rank))
        out.append((info, torch.from_numpy(blob).to("cuda")))
    return out
