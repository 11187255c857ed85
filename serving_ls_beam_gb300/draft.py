"""Decoding with a tree of drafted tokens per row: the attention of every layer, the choice and the
commit of one step, over device-resident caches.

One step evaluates ``nodes`` tokens per row at once: node 0 is the token chosen by the step before,
the others guess what follows it (``parent`` says after which node; -2 leaves a place empty).  For
each layer the caller projects queries, keys and values and calls ``self_attention`` (the row's
cache and the node's own branch, ``ls_tree_attention``) and, with an encoder, ``cross_attention``
(``ls_cross_attention``: every row of a sentence reads its encoder states).  ``finish`` then takes
the nodes' logits, chooses a token after every node (``ls_sample`` with one candidate), finds the
branch those choices confirm and appends its keys and values to the cache of every layer
(``ls_tree_commit``).  The result is that of decoding one token at a time; with ``nodes`` = 1 it
is that.  Every row decodes greedily for itself, those of one sentence too: there is no selection
among beams here (``loop.py`` has it).

Everything stays on the GPU and every buffer is allocated once, so that a step can be captured in a
CUDA graph (the memory-reuse rule of the LightSeq inference article, 31duo.com, itemid-283120, as
in ``loop.py``; the two sets of lengths alternate, so capture two steps).

``stream`` (a stream of torch's or its handle; torch's current one by default) is where a call's work
goes, all of it.  The caller orders that stream behind the inputs and keeps them until it has passed.
``reset`` works on the current stream.
"""
from __future__ import annotations

import contextlib

import torch

from . import (check, ls_cross_attention, ls_cross_attention_workspace_size, ls_sample, ls_sample_workspace_size,
               ls_tree_attention, ls_tree_attention_workspace_size, ls_tree_commit, ls_workspace_init)


def _torch_on(stream, device):
    """Torch's own operations on the stream that the library's calls are given."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


class DraftTreeDecoder:
    def __init__(self, layers: int, rows: int, nodes: int, heads: int, kv_heads: int, head_dim: int, max_len: int,
                 vocab: int, eos_id: int, dtype=torch.float16, device="cuda", beams: int = 1):
        """rows sequences of up to max_len positions; beams: rows per sentence of the encoder (rows = batch * beams)."""
        dev = torch.device(device)
        if rows % beams:
            raise ValueError("rows must be a multiple of beams")
        self.layers, self.rows, self.nodes, self.heads, self.kv_heads = layers, rows, nodes, heads, kv_heads
        self.head_dim, self.max_len, self.vocab, self.eos_id, self.beams = head_dim, max_len, vocab, eos_id, beams

        def empty(*shape, dt=dtype):
            return torch.empty(shape, dtype=dt, device=dev)

        def words(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=dev)

        self.cache_key = empty(layers, rows, kv_heads, max_len, head_dim)
        self.cache_value = empty(layers, rows, kv_heads, max_len, head_dim)
        self.draft_key = empty(layers, rows, nodes, kv_heads, head_dim)
        self.draft_value = empty(layers, rows, nodes, kv_heads, head_dim)
        self.lengths = [words(rows), words(rows)]  # read by a step / written by it
        self.finished = [torch.zeros(rows, dtype=torch.uint8, device=dev) for _ in range(2)]
        self.path, self.count, self.next_token = words(rows, nodes), words(rows), words(rows)
        self.target = words(rows, nodes)
        self.greedy_u = torch.zeros(rows * nodes, dtype=torch.float32, device=dev)
        self.attended = empty(rows, nodes, heads, head_dim)
        self.cur = 0
        self.encoder = None  # per layer (keys, values) [batch, kv_heads, max_src, head_dim], and the lengths
        size = ls_tree_attention_workspace_size(rows, nodes, heads, kv_heads, max_len, head_dim)
        cross = ls_cross_attention_workspace_size(rows // beams, beams, nodes, heads, kv_heads, 1, head_dim)
        self.workspace = torch.empty(max(size, cross), dtype=torch.uint8, device=dev)
        check(ls_workspace_init(self.workspace), "ls_workspace_init")
        self.sample_workspace = torch.empty(ls_sample_workspace_size(rows * nodes, 1, vocab), dtype=torch.uint8, device=dev)
        check(ls_workspace_init(self.sample_workspace), "ls_workspace_init")

    def reset(self, encoder=None, src_len=None):
        """Start new sequences: empty caches; encoder: a (keys, values) pair per layer, src_len [batch] int32."""
        self.cur = 0
        for t in self.lengths + self.finished:
            t.zero_()
        self.encoder, self.src_len = encoder, src_len

    def length(self) -> torch.Tensor:
        """Positions in each row's cache [rows] int32 (positions of the next step's node 0)."""
        return self.lengths[self.cur]

    def self_attention(self, layer: int, q, key, value, parent, stream=None) -> torch.Tensor:
        """q [rows, nodes, heads, head_dim], key and value [rows, nodes, kv_heads, head_dim] of this layer's nodes, parent
        [rows, nodes] int32.  Returns a buffer that the next attention overwrites."""
        with _torch_on(stream, self.draft_key.device):
            self.draft_key[layer].copy_(key)
            self.draft_value[layer].copy_(value)
        check(ls_tree_attention(q, self.cache_key[layer], self.cache_value[layer], self.lengths[self.cur],
                                self.draft_key[layer], self.draft_value[layer], parent, self.attended, self.workspace,
                                stream=stream), "ls_tree_attention")
        return self.attended

    def cross_attention(self, layer: int, q, stream=None) -> torch.Tensor:
        """q [rows, nodes, heads, head_dim] over the encoder's states of each row's sentence."""
        keys, values = self.encoder[layer]
        shape = (self.rows // self.beams, self.beams, self.nodes, self.heads, self.head_dim)
        check(ls_cross_attention(q.view(shape), keys, values, self.src_len, self.attended.view(shape), self.workspace,
                                 stream=stream), "ls_cross_attention")
        return self.attended

    def finish(self, logits, token, parent, stream=None) -> torch.Tensor:
        """logits [rows, nodes, vocab], token and parent [rows, nodes] int32: choose, confirm, append.  Returns the next
        token of every row [rows] int32; path and count tell what was appended, finished[cur] whose search has ended."""
        s, n = self.cur, 1 - self.cur
        check(ls_sample(logits.view(self.rows * self.nodes, self.vocab), None, self.greedy_u, 1, 1.0,
                        self.target.view(-1), None, self.sample_workspace, stream), "ls_sample")
        check(ls_tree_commit(self.cache_key, self.cache_value, self.lengths[s], self.draft_key, self.draft_value, parent,
                             token, self.target, self.finished[s], self.eos_id, self.lengths[n], self.path, self.count,
                             self.next_token, self.finished[n], self.workspace, stream), "ls_tree_commit")
        self.cur = n
        return self.next_token
