"""Decoding over a cache in pages: rows of any lengths share one pool of pages, held as they are or in 8 bits.

One step evaluates one token per row.  For each layer the caller projects queries, keys and values and calls
``attention``: the token's keys and values go to the row's next position (``ls_paged_write``, quantised where the
pages have 8 bits) and the queries read the row's positions with it (``ls_paged_attention``).  ``finish`` takes the
logits and draws every row's next token with settings of its own (``ls_sample_filtered``).  A row that draws
``eos_id``, or finds nothing to draw (-1), is finished: it writes and advances no more, its token is ``eos_id`` from
then on, and its queries read what it holds until it is released.

A sequence takes an idle row, with length 0, by that row's first ``reserve``, and leaves it by ``release``.  An idle row
takes part in every step with nothing: it writes nothing, its attention is zeros and its token ``eos_id``.  A prompt is
stored layer by layer with ``store`` and counted once with ``advance``, before the next step; ``restore`` gives a
layer's cache back as dense tensors (``ls_paged_read``).  Which pages a row has is kept on the host: ``reserve`` before
the positions are written, ``release`` when the sequence is done.

The tables, lengths and settings are tensors of fixed places, so that a step can be captured in a CUDA graph (the
memory-reuse rule of the LightSeq inference article, 31duo.com, itemid-283120, as in ``loop.py``) and replayed after
``reserve`` and ``release``, which write to them in stream order.  ``stream`` (a stream of torch's or its handle; torch's
current one by default) is where a call's work goes, all of it.  The caller orders that stream behind the inputs.
"""
from __future__ import annotations

import torch

from . import (check, ls_paged_attention, ls_paged_attention_workspace_size, ls_paged_read, ls_paged_write, ls_pages,
               ls_sample_filtered, ls_workspace_init)
from .draft import _torch_on


class PagedDecoder:
    def __init__(self, layers: int, rows: int, heads: int, kv_heads: int, head_dim: int, page_size: int, num_pages: int,
                 max_pages: int, eos_id: int, dtype=torch.float16, cache_dtype=None, device="cuda"):
        """rows sequences of up to max_pages pages each, of num_pages in all; cache_dtype: dtype (the default),
        torch.float8_e4m3fn or torch.int8."""
        dev = torch.device(device)
        cache_dtype = dtype if cache_dtype is None else cache_dtype
        self.layers, self.rows, self.heads, self.kv_heads, self.head_dim = layers, rows, heads, kv_heads, head_dim
        self.page_size, self.num_pages, self.max_pages, self.eos_id = page_size, num_pages, max_pages, eos_id
        shape = (layers, num_pages, kv_heads, page_size, head_dim)
        coded = cache_dtype in (torch.float8_e4m3fn, torch.int8)

        def words(*s):
            return torch.zeros(s, dtype=torch.int32, device=dev)

        self.key, self.value = (torch.empty(shape, dtype=cache_dtype, device=dev) for _ in range(2))
        self.key_scale, self.value_scale = (torch.empty(shape[:4], device=dev) if coded else None for _ in range(2))
        self.table = torch.full((rows, max_pages), -1, dtype=torch.int32, device=dev)
        self.pages = [ls_pages(self.key[i], self.value[i], self.table, self.key_scale[i] if coded else None,
                               self.value_scale[i] if coded else None) for i in range(layers)]
        self.length = words(rows)      # positions held
        self.live = words(rows)        # 1: a sequence that goes on; 0: finished, or none
        self.seen = words(rows)        # positions with the step's own
        self.next_token = words(rows)
        self.logprob = torch.zeros(rows, device=dev)
        self.attended = torch.empty((rows, heads, head_dim), dtype=dtype, device=dev)
        self.workspace = torch.empty(ls_paged_attention_workspace_size(rows, heads, kv_heads, head_dim), dtype=torch.uint8,
                                     device=dev)
        check(ls_workspace_init(self.workspace), "ls_workspace_init")
        self.free = list(range(num_pages - 1, -1, -1))
        self.held = [[] for _ in range(rows)]

    def reserve(self, row: int, positions: int, stream=None) -> None:
        """Pages for the first `positions` positions of a row; a sequence begins with the row's first page.  ValueError where the
        row or the pool has no room; nothing is taken then."""
        need = -(-positions // self.page_size) - len(self.held[row])
        if need <= 0:
            return
        if len(self.held[row]) + need > self.max_pages:
            raise ValueError(f"row {row}: {positions} positions need more than max_pages = {self.max_pages} pages")
        if need > len(self.free):
            raise ValueError(f"row {row}: {need} pages needed, {len(self.free)} left")
        first = len(self.held[row])
        new = [self.free.pop() for _ in range(need)]
        self.held[row] += new
        with _torch_on(stream, self.table.device):
            self.table[row, first:first + need].copy_(torch.tensor(new, dtype=torch.int32))
            if first == 0:
                self.live[row] = 1
                self.seen[row] = 1

    def release(self, row: int, stream=None) -> None:
        """The row's pages back to the pool; the row is idle until it gets pages again."""
        self.free += reversed(self.held[row])
        self.held[row] = []
        with _torch_on(stream, self.table.device):
            self.table[row].fill_(-1)
            self.length[row] = 0
            self.live[row] = 0
            self.seen[row] = 0

    def store(self, layer: int, key, value, count=None, stream=None) -> None:
        """A prompt's keys and values [rows, tokens, kv_heads, head_dim] behind what the rows hold, the first count [rows]
        int32 of each row (None: all, of the live rows); the lengths stay until advance."""
        if count is None:
            with _torch_on(stream, self.table.device):
                count = self.live * key.shape[1]
        check(ls_paged_write(key, value, self.length, count, self.pages[layer], self.workspace, stream), "ls_paged_write")

    def advance(self, count, stream=None) -> None:
        """Lengths of the live rows after a prompt has been stored in every layer: count [rows] int32, or a number for all."""
        with _torch_on(stream, self.table.device):
            self.length.add_(self.live * count)
            torch.add(self.length, self.live, out=self.seen)

    def restore(self, layer: int, key, value, stream=None) -> None:
        """The layer's cache into key, value [rows, tokens, kv_heads, head_dim]; what lies behind a row's length stays."""
        check(ls_paged_read(self.pages[layer], None, self.length, key, value, self.workspace, stream), "ls_paged_read")

    def attention(self, layer: int, q, key, value, stream=None) -> torch.Tensor:
        """q [rows, heads, head_dim], key and value [rows, kv_heads, head_dim] of the step's tokens.  Returns a buffer that the
        next attention overwrites."""
        check(ls_paged_write(key.unsqueeze(1), value.unsqueeze(1), self.length, self.live, self.pages[layer], self.workspace,
                             stream), "ls_paged_write")
        check(ls_paged_attention(q, self.pages[layer], self.seen, self.attended, self.workspace, stream=stream),
              "ls_paged_attention")
        return self.attended

    def finish(self, logits, u, temperature=None, top_k=None, top_p=None, min_p=None, stream=None) -> torch.Tensor:
        """logits [rows, vocab], u [rows] f32 and the rows' settings (None: off): the next token of every row [rows] int32
        (logprob: of its probability; of rows that are not live it says nothing), and the rows' lengths advanced."""
        check(ls_sample_filtered(logits, None, u, temperature, top_k, top_p, min_p, self.next_token, self.logprob,
                                 self.workspace, stream), "ls_sample_filtered")
        with _torch_on(stream, self.table.device):
            self.next_token.masked_fill_(self.live == 0, self.eos_id)
            self.length.add_(self.live)
            self.live.mul_((self.next_token != self.eos_id) & (self.next_token >= 0))
            torch.add(self.length, self.live, out=self.seen)
        return self.next_token
