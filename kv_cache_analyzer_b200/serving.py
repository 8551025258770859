"""Several generations over one page pool: the cache step of each layer for a
batch of images and videos of different sizes.

A generation keeps its whole sequence cached and refreshes only its due tokens
per step; a streamed one also grows.  ``PagedBatch`` owns the pool and hands its
pages out (host bookkeeping; the device sees page tables, lengths and row
offsets), and one step of all generations is two calls:

  paged_append     the due tokens' K (rotated on the way) and V into their
                   pages, their queries rotated in the same launch
  paged_attention  the due queries of every generation over its own pages

so small due sets of several generations fill the GPU together.  ``plan`` makes
the device lists of a batch; everything a step reads is in device memory when it
returns, so ``step`` can be captured as a CUDA graph (keep the plan for as long
as the graph, and capture again once one of its generations grew or closed).
"""
from __future__ import annotations

import contextlib
import operator
from dataclasses import dataclass

import torch

from . import _torch_stream
from .paged import Rope, page_pool, paged_append, paged_attention, rope_table


@dataclass(frozen=True)
class BatchPlan:
    """The device lists of one batch of generations, and what the host knows of it."""
    lists: dict             # page_table, seq_lens, cu_rows
    grids: torch.Tensor | None
    max_rows: int
    max_len: int
    n_rows: int
    gens: tuple             # (generation, its tokens) as planned


class PagedBatch:
    """Page pool of `n_pages` pages of `page_size` tokens, shared by the open
    generations: K and V pages per layer, one page table for all layers.  heads
    query heads attend over kv_heads K/V heads of size d; with a rope, K and Q
    are rotated by their token's position (on the rope's grid, or on each
    generation's own, see ``open``).  All work is launched on `stream`."""

    def __init__(self, *, n_pages: int, page_size: int, heads: int, d: int, kv_heads: int | None = None,
                 rope: Rope | None = None, layers: int = 1, head_major: bool = False, device="cuda", stream=None):
        self.page_size, self.heads, self.d = page_size, heads, d
        self.kv_heads = heads if kv_heads is None else kv_heads
        self.dev, self.stream = torch.device(device), stream
        if layers < 1:
            raise ValueError(f"layers must be at least 1, got {layers}")
        with self._on_stream():
            self.layers = [page_pool(n_pages, page_size, self.kv_heads, d, head_major, self.dev)
                           for _ in range(layers)]
        self.k_pages, self.v_pages = self.layers[0]
        self.rope = rope
        self.table = None if rope is None else rope_table(rope, stream=stream, device=self.dev)
        self._free = list(range(n_pages))[::-1]
        self._gens: dict[int, dict] = {}
        self._next = 0

    def _on_stream(self):
        """Memory made here belongs to the batch's stream: it is reused behind the steps that read it."""
        return contextlib.nullcontext() if self.stream is None else torch.cuda.stream(_torch_stream(self.stream))

    # ------------------------------------------------------------------ pages
    @property
    def free_pages(self) -> int:
        return len(self._free)

    def open(self, n_tokens: int, grid: tuple | None = None) -> int:
        """A new generation of n_tokens cached positions (their pages are
        reserved now; their contents are whatever the pages held until they
        are appended).  grid: its (rows, columns) of tokens, if it differs from
        the rope's."""
        g = dict(pages=[], tokens=0, grid=grid)
        # (before the batch knows of it: a refused generation leaves nothing)
        self._reserve(g, operator.index(n_tokens))
        gen = self._next
        self._next += 1
        self._gens[gen] = g
        return gen

    def extend(self, gen: int, n_tokens: int) -> None:
        """The generation grows to n_tokens cached positions."""
        g = self._gens[gen]
        n_tokens = operator.index(n_tokens)
        if n_tokens < g["tokens"]:
            raise ValueError(f"generation {gen} has {g['tokens']} tokens, cannot shrink to {n_tokens}")
        self._reserve(g, n_tokens)

    def _reserve(self, g: dict, n_tokens: int) -> None:
        if n_tokens < 0:
            raise ValueError(f"a generation cannot have {n_tokens} tokens")
        need = -(-n_tokens // self.page_size) - len(g["pages"])
        if need > len(self._free):
            raise RuntimeError(f"page pool exhausted: {need} pages needed, {len(self._free)} free")
        g["pages"] += [self._free.pop() for _ in range(need)]
        g["tokens"] = n_tokens

    def close(self, gen: int) -> None:
        """Give the generation's pages back (after the work on them is enqueued:
        the next owner's appends follow it on the same stream)."""
        self._free += self._gens.pop(gen)["pages"][::-1]

    # ------------------------------------------------------------------ step
    def plan(self, rows: list[tuple[int, int]]) -> BatchPlan:
        """The lists of a batch: (generation, due rows) in the order of the
        packed rows.  It holds until one of its generations grows or closes."""
        if not rows:
            raise ValueError("a batch needs at least one generation")
        if len({g for g, _ in rows}) != len(rows):
            raise ValueError("a generation appears once in a batch")
        counts = [n for _, n in rows]
        if min(counts) < 0:
            raise ValueError(f"row counts must not be negative, got {counts}")
        gens = [self._gens[g] for g, _ in rows]
        width = max(1, max(len(g["pages"]) for g in gens))
        table = torch.zeros(len(rows), width, dtype=torch.int32)
        for s, g in enumerate(gens):
            table[s, :len(g["pages"])] = torch.tensor(g["pages"], dtype=torch.int32)
        cu = torch.zeros(len(rows) + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(counts, dtype=torch.int32).cumsum(0)
        lens = torch.tensor([g["tokens"] for g in gens], dtype=torch.int32)
        grids = None
        if self.rope is not None and any(g["grid"] is not None for g in gens):
            grids = torch.tensor([g["grid"] or self.rope.grid for g in gens], dtype=torch.int32)
        with self._on_stream():
            lists = dict(page_table=table.to(self.dev), seq_lens=lens.to(self.dev), cu_rows=cu.to(self.dev))
            grids = None if grids is None else grids.to(self.dev)
        return BatchPlan(lists, grids, max(counts), int(lens.max()), sum(counts),
                         tuple((gen, g["tokens"]) for (gen, _), g in zip(rows, gens)))

    def step(self, plan: BatchPlan, q, k, v, pos, limits=None, out=None, layer: int = 0):
        """One layer's step of a planned batch: k, v [rows][kv_heads][d] of
        the due tokens pos (int32, rising within a generation) go to their
        pages, q [rows][heads][d] attends.  limits: positions each row sees
        (None: all).  Returns out [rows][heads][d]."""
        for gen, tokens in plan.gens:
            if gen not in self._gens or self._gens[gen]["tokens"] != tokens:
                raise ValueError(f"generation {gen} grew or closed after the plan was made")
        if pos.numel() != plan.n_rows:
            raise ValueError(f"the plan has {plan.n_rows} rows, got {pos.numel()}")
        k_pages, v_pages = self.layers[layer]
        q_rot = paged_append(k, v, pos, k_pages, v_pages, **plan.lists, rope=self.rope, table=self.table,
                             q=q, grids=plan.grids, stream=self.stream)
        return paged_attention(q_rot, k_pages, v_pages, **plan.lists, limits=limits, out=out,
                               max_rows=plan.max_rows, max_len=plan.max_len, stream=self.stream)
