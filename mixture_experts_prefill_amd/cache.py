"""A paged key-value cache for a batch of sequences, and the attention over it.

Owns one buffer a layer, the page tables, lengths and free pages that all
layers share, and the plan of the current step.  Lengths and tables live on the
GPU and advance there; no call reads them back, so a step may be captured into
a graph and replayed.  The arithmetic is in libmoe.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (moe_attention_decode, moe_attention_prefill, moe_attention_workspace_bytes, moe_kv_append,
               moe_kv_layout_make, moe_kv_plan_step)
from .matrix import _allocating_on


class MoeCache:
    def __init__(self, layers: int, n: int, rows: int, pages: int, page: int, heads: int, head: int, heads_q: int,
                 max_pages: int, dtype: torch.dtype = torch.bfloat16, device: str = "cuda"):
        """A cache of `pages` pages of `page` tokens a layer for n sequences of at most max_pages pages and steps of
        at most `rows` rows; bfloat16 or float8_e4m3fn.  The calls of one cache share a workspace: they are made on
        one stream, or ordered by events."""
        self.layout = moe_kv_layout_make(pages, page, heads, head, dtype)
        self.n, self.rows, self.heads_q = n, rows, heads_q
        self.cache = [torch.empty(self.layout.bytes, dtype=torch.uint8, device=device) for _ in range(layers)]

        def ints(*shape):
            return torch.zeros(*shape, dtype=torch.int32, device=device)

        self.table, self.length = ints(n, max_pages), ints(n)
        self.free_pages = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device)  # page 0 on top
        self.free_n = torch.full((1,), pages, dtype=torch.int32, device=device)
        self.starts, self.positions, self.slots, self.lacking = ints(n + 1), ints(rows), ints(rows), ints(1)
        self.before = torch.cat([self.length, self.free_n])  # lengths and free pages before the step
        need = moe_attention_workspace_bytes(rows, n, heads_q, self.layout)
        if not need:
            raise ValueError(f"no attention of {rows} rows of {n} sequences with {heads_q} query heads on this cache")
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)

    def plan(self, grow: torch.Tensor, stream=None, again: bool = False) -> None:
        """Start a step in which sequence s gains grow[s] rows (int32 [n]; -1: it is finished, and its place may be
        used by another one).  lacking is then the number of rows without a slot, 0 in a good step: they are the last
        of their sequences, are not appended, and attention gives 0 for them.  again: the step takes the place of the
        one planned last, which lacked pages, say; where that one was appended already, its rows are appended anew."""
        moe_kv_plan_step(self.length, grow, self.layout, self.table, self.free_pages, self.free_n, self.before,
                         self.starts, self.positions, self.slots, self.lacking, again, stream)

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, rope: Optional[torch.Tensor] = None,
               q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None, stream=None):
        """The step's rows k and v into a layer's cache; with rope also q turned, into q_out or a new tensor, which
        is returned."""
        t = k.shape[0]
        if q is not None and q_out is None:
            with _allocating_on(stream, q.device):
                q_out = torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)  # rows without a slot stay 0
        moe_kv_append(k, v, self.layout, self.cache[layer], self.slots[:t], None if rope is None else self.positions[:t],
                      rope, q, q_out, stream)
        return q_out

    def attend(self, layer: int, q: torch.Tensor, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               single: bool = False, stream=None) -> torch.Tensor:
        """Causal attention of the step's rows q [t, heads_q * head], into `out` or a new tensor whose rows past the
        step's are 0, as those without a slot are.  single: no sequence has more than one row in this step (one new token each)."""
        if out is None:
            with _allocating_on(stream, q.device):
                out = torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
        scale = self.layout.head ** -0.5 if scale is None else scale
        if single:
            moe_attention_decode(q, self.layout, self.cache[layer], self.table, self.length, scale, out, self.workspace,
                                 self.starts, stream, self.before[:self.n])
        else:
            moe_attention_prefill(q, self.starts, self.layout, self.cache[layer], self.table, self.length, scale, out,
                                  self.workspace, stream, self.before[:self.n])
        return out
