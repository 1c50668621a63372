"""A batch of sequences over one paged key / value cache: the dense grouped-head
layer that stands beside the compressed ones of `stack.py`.

A driver over the C-ABI entry points: it owns the pages, the block table and
the lengths of one layer (torch allocations) and calls paged_append,
prompt_attn and paged_decode_attn in order.  No arithmetic happens here.
"""
from __future__ import annotations

from . import (OP_PAGED_DECODE, OP_PROMPT_ATTN, GqaParams, empty_paged, gqa_workspace_size, paged_append,
               paged_decode_attn, prompt_attn)


class PagedLayer:
    """Cache of `n_seq` sequences that share `n_pages` pages; a sequence holds at
    most `max_pages` of them."""

    def __init__(self, p: GqaParams, n_seq: int, n_pages: int, max_pages: int, inv_freq=None, device="cuda"):
        import torch
        self.p, self.n_seq, self.inv_freq = p, n_seq, inv_freq
        self.k_cache, self.v_cache = empty_paged(p, n_pages, device)
        self.table = torch.full((n_seq, max_pages), -1, dtype=torch.int32, device=device)
        self.lens = [0] * n_seq                    # tokens of each sequence, host side
        self.pos = torch.full((n_seq,), -1, dtype=torch.int64, device=device)
        self._free = list(range(n_pages - 1, -1, -1))
        self._held = [[] for _ in range(n_seq)]
        # decode workspace, allocated once so that decode steps can be captured in a graph
        self.ws = torch.empty(gqa_workspace_size(p, OP_PAGED_DECODE, n_seq, n_seq, max_pages * p.page_size),
                              dtype=torch.uint8, device=device)

    def _missing(self, s: int, n: int) -> int:
        """Pages that sequence s lacks for n more tokens."""
        return max(-(-(self.lens[s] + n) // self.p.page_size) - len(self._held[s]), 0)

    def _check_room(self, wants):
        """Raise, before any page is taken, unless the pool and the table hold n more tokens of each
        sequence s, for all (s, n)."""
        free = len(self._free)
        for s, n in wants:
            need = self._missing(s, n)
            free -= need
            if free < 0 or len(self._held[s]) + need > self.table.shape[1]:
                raise RuntimeError(f"sequence {s}: no room for {n} more tokens")

    def reserve(self, s: int, n: int):
        """Pages for the next n tokens of sequence s (raises when the pool or the table is full)."""
        self._check_room([(s, n)])
        self._take(s, n)

    def _take(self, s: int, n: int):
        need, first = self._missing(s, n), len(self._held[s])
        if need == 0:
            return
        import torch
        self._held[s] += [self._free.pop() for _ in range(need)]
        self.table[s, first:first + need] = torch.tensor(self._held[s][first:], dtype=torch.int32)

    def release(self, s: int):
        """Give the pages of sequence s back; it is empty afterwards."""
        self._free += self._held[s]
        self._held[s], self.lens[s] = [], 0
        self.table[s] = -1
        self.pos[s] = -1

    def prefill(self, lens, q, k, v, sinks, out):
        """The whole prompts of empty sequences: lens[s] tokens of sequence s (0: none), packed
        in q [n][H][d], k, v [n][HK][d]; out [n][H][d].  Rows from sum(lens) on are padding.  The
        rotated queries and keys live until the attention has read them."""
        import torch
        if len(lens) != self.n_seq or any(n < 0 for n in lens):
            raise ValueError(f"lens must be {self.n_seq} lengths of at least 0, got {list(lens)}")
        if any(n and self.lens[s] for s, n in enumerate(lens)):
            raise ValueError("a prompt for a sequence that holds tokens: release it first")
        if sum(lens) > q.shape[0]:
            raise ValueError(f"prompts of {sum(lens)} tokens in {q.shape[0]} rows")
        self._check_room(enumerate(lens))
        for s, n in enumerate(lens):
            self._take(s, n)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        dev, n = q.device, q.shape[0]
        cu = torch.tensor(cu, dtype=torch.int32, device=dev)
        pos0 = torch.zeros(self.n_seq, dtype=torch.int64, device=dev)
        qr, kr = (torch.empty(t.shape, dtype=t.dtype, device=dev) for t in (q, k))
        paged_append(self.p, self.n_seq, n, cu, pos0, q, k, v, self.inv_freq, qr, kr, self.k_cache, self.v_cache,
                     self.table)
        ws = torch.empty(gqa_workspace_size(self.p, OP_PROMPT_ATTN, self.n_seq, n, 0), dtype=torch.uint8, device=dev)
        prompt_attn(self.p, self.n_seq, qr, kr, v, cu, cu, sinks, out, ws)
        self.lens = [a + n for a, n in zip(self.lens, lens)]
        self.pos.copy_(torch.tensor([n - 1 for n in self.lens], dtype=torch.int64))

    def advance(self, active=None):
        """Host side of a decode step: room for one more token of each active sequence (all
        that hold tokens, when not given; each named once), whose positions move on by one.  A
        sequence left out is at position -1 in this step."""
        import torch
        active = [s for s, n in enumerate(self.lens) if n] if active is None else list(active)
        if len(set(active)) != len(active) or any(not 0 <= s < self.n_seq for s in active):
            raise ValueError(f"active must name sequences 0 to {self.n_seq - 1}, each once, got {active}")
        self._check_room((s, 1) for s in active)  # a full pool leaves everything as it was
        for s in active:
            self._take(s, 1)
        for s in active:
            self.lens[s] += 1
        pos = [-1] * self.n_seq
        for s in active:
            pos[s] = self.lens[s] - 1
        self.pos.copy_(torch.tensor(pos, dtype=torch.int64))

    def step(self, q, k, v, sinks, out, q_rot):
        """Device side of a decode step, after advance(): append the new token of each sequence
        and attend it.  q, out, q_rot [n_seq][H][d], k, v [n_seq][HK][d]; q_rot receives the
        rotated queries.  Rows of sequences that are left out: 0.  Can be captured in a graph
        and replayed after further calls of advance()."""
        paged_append(self.p, self.n_seq, self.n_seq, None, self.pos, q, k, v, self.inv_freq, q_rot, None, self.k_cache,
                     self.v_cache, self.table)
        paged_decode_attn(self.p, self.n_seq, q_rot, self.k_cache, self.v_cache, self.table, self.pos, sinks, out, self.ws)

    def decode(self, q, k, v, sinks, out, active=None):
        """One decode step: advance(), then step()."""
        import torch
        self.advance(active)
        self.step(q, k, v, sinks, out, torch.empty(q.shape, dtype=q.dtype, device=q.device))
