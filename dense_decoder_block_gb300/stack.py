"""A decoder-only stack sequenced from the library's calls.

"How Llama 3.1 Generates the Next Token" (the transformer blocks, Unembedding,
Sampling) and "Llama 3.1 70B" (Token embedding, Transformer layer, LM head):
token ids are embedded, pass through L decoder blocks, and the last position's
hidden state goes through the final RMSNorm and the LM head; the next id is the
greedy choice.  Every arithmetic step runs in the library's kernels
(llama_embed, llama_block_prefill / llama_block_decode_devpos,
llama_lmhead_argmax); this module only orders the calls and owns the per-layer
KV caches and the scratch buffers, all allocated once.
"""
from __future__ import annotations

import contextlib
from typing import Callable, Dict, List, Optional, Sequence, Tuple

import torch

from . import (KVCache, LlamaBlock, PagedCache, PagedCacheList, llama_beam_reorder, llama_beam_select,
               llama_beam_select_workspace_bytes, llama_embed, llama_lmhead_argmax, llama_lmhead_workspace_bytes,
               llama_paged_plan, llama_paged_release, llama_paged_store)


class LlamaStack:
    """L blocks of one shape plus embedding and head, for `batch` sequences of up to
    `max_seq` positions.  Weights are borrowed (device tensors, [out, in] bf16)."""

    def __init__(self, dims, layers: Sequence[Tuple[Dict[str, torch.Tensor], Dict[str, torch.Tensor]]],
                 w_embed: torch.Tensor, g_final: torch.Tensor, w_out: torch.Tensor, batch: int, max_seq: int,
                 prefill_tokens: int):
        dev = w_embed.device
        dt = w_embed.dtype
        self.dims, self.batch, self.max_seq, self.prefill_tokens = dims, batch, max_seq, prefill_tokens
        self.vocab = w_embed.shape[0]
        self.w_embed, self.g_final, self.w_out = w_embed, g_final, w_out
        self.blocks: List[LlamaBlock] = [LlamaBlock(dims, w, g, max_seq) for w, g in layers]
        shape = (batch, dims.n_kv_heads, max_seq, dims.head_dim)
        self.caches: List[KVCache] = [KVCache(torch.zeros(shape, dtype=dt, device=dev),
                                              torch.zeros(shape, dtype=dt, device=dev)) for _ in layers]
        ws_bytes = max(self.blocks[0].workspace_bytes(batch, prefill_tokens), self.blocks[0].workspace_bytes(batch, 1))
        self.ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        # activations ping-pong between two flat buffers large enough for the prefill
        self.act = [torch.empty(batch * prefill_tokens * dims.d_model, dtype=dt, device=dev) for _ in range(2)]
        self.head_ws = torch.empty(llama_lmhead_workspace_bytes(batch, dims.d_model, self.vocab), dtype=torch.uint8,
                                   device=dev)
        self.logits = torch.empty(batch, self.vocab, dtype=torch.float32, device=dev)
        self.ids = torch.zeros(batch, dtype=torch.int32, device=dev)   # the chosen ids (decode feeds them back)
        self.pos = torch.zeros(1, dtype=torch.int32, device=dev)       # the decode position, on the device
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)       # out-of-range ids from llama_embed
        # prefill may go to another stream than the one that filled all this
        torch.cuda.current_stream(dev).synchronize()

    @staticmethod
    def _on(stream):
        # the position counter is updated on the stream the library calls were issued on
        return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()

    def _acts(self, T: int):
        n = self.batch * T * self.dims.d_model
        return [a[:n].view(self.batch, T, self.dims.d_model) for a in self.act]

    def _head(self, x: torch.Tensor, T: int, stream) -> None:
        # the last position of each sequence: rows T-1, 2T-1, ... of x [B, T, d], i.e.
        # B rows T * d elements apart starting at row T-1
        last = x.view(-1)[(T - 1) * self.dims.d_model:]
        llama_lmhead_argmax(last, self.batch, T * self.dims.d_model, self.g_final, self.w_out, self.vocab,
                            self.dims.d_model, self.dims.eps, self.ids, self.logits, self.head_ws,
                            self.head_ws.numel(), stream)

    def prefill(self, ids: torch.Tensor, stream: Optional[torch.cuda.Stream] = None,
                on_layer: Optional[Callable[[int, torch.Tensor], None]] = None) -> None:
        """ids [B, T] int32 on the device, positions 0..T-1.  Leaves the logits of the
        last position in self.logits, the greedy ids in self.ids, and self.pos = T.
        ``on_layer(l, h)``, if given, sees the embedding (l = -1) and each block's
        output h [B, T, d] as soon as its call is enqueued (for inspection)."""
        B, T = ids.shape
        assert B == self.batch and T <= self.prefill_tokens
        x, y = self._acts(T)
        llama_embed(ids, B * T, self.w_embed, self.vocab, self.dims.d_model, x, self.err, stream)
        if on_layer:
            on_layer(-1, x)
        for l, (blk, kv) in enumerate(zip(self.blocks, self.caches)):
            blk.prefill(x, kv, y, self.ws, stream)
            if on_layer:
                on_layer(l, y)
            x, y = y, x
        self._head(x, T, stream)
        with self._on(stream):
            self.pos.fill_(T)

    def decode_step(self, stream: Optional[torch.cuda.Stream] = None,
                    on_layer: Optional[Callable[[int, torch.Tensor], None]] = None) -> None:
        """One token for every sequence at position self.pos (on the device): embeds
        self.ids, runs the blocks, writes the next ids into self.ids and advances
        self.pos.  Capturable in a CUDA graph (nothing is read on the host) when
        ``on_layer`` (as in prefill) is not given."""
        x, y = self._acts(1)
        llama_embed(self.ids, self.batch, self.w_embed, self.vocab, self.dims.d_model, x, self.err, stream)
        if on_layer:
            on_layer(-1, x)
        for l, (blk, kv) in enumerate(zip(self.blocks, self.caches)):
            blk.decode_devpos(x, kv, self.pos, y, self.ws, stream)
            if on_layer:
                on_layer(l, y)
            x, y = y, x
        self._head(x, 1, stream)
        with self._on(stream):
            self.pos.add_(1)

    def poll_error(self) -> int:
        for blk in self.blocks:
            rc = blk.poll_error()
            if rc:
                return rc
        return 0


class BeamSearch:
    """Beam search on a stack: `beams` continuations of each of the stack's requests, at most `max_new` tokens,
    on a paged cache.  A request's beams share the full pages of their common past; each owns the pages from its
    first unfilled one on.  Row g * beams + k of every tensor is beam k of request g; groups * beams <= 32.

        bs = BeamSearch(stack, beams=4, max_new=64, eos=2)
        bs.begin(ids)                  # prompts [requests, T]: prefill, pages, the first tokens
        for _ in range(63):
            bs.step()                  # one more token per beam (capturable in a CUDA graph)
        tokens, scores = bs.sequences()
        bs.end()                       # the pages go back to the pool

    eos < 0: no beam ends.  A beam that ended keeps its score and repeats eos.  The calls take any stream; those of
    one search are ordered by the caller (one stream, or events)."""

    def __init__(self, stack: LlamaStack, beams: int, max_new: int, eos: int = -1, page_size: int = 16):
        dims, dev, dt = stack.dims, stack.w_embed.device, stack.w_embed.dtype
        groups = stack.batch
        rows = groups * beams
        if beams < 1 or rows > 32:
            raise ValueError("requests x beams must be 1 to 32 rows")
        group = dims.n_heads // dims.n_kv_heads
        if dt != torch.bfloat16 or group > 64 or 128 % group:
            raise ValueError("paged steps take bf16 blocks whose query heads per KV head divide 128 (at most 64)")
        if beams > stack.vocab:
            raise ValueError("more beams than tokens to choose from")
        if max_new < 1 or max_new >= stack.max_seq:
            raise ValueError("max_new must leave room for a prompt in the stack's max_seq")
        # what a call would refuse in the middle of a search, with pages taken and positions advanced
        if eos >= stack.vocab:
            raise ValueError("eos must be a token of the stack's vocabulary, or negative")
        if stack.vocab > 1 << 20:
            raise ValueError("the selection takes at most 2^20 tokens")
        if not 16 <= page_size <= 1024 or page_size & (page_size - 1):
            raise ValueError("page_size must be a power of two in 16 .. 1024")
        if len(stack.blocks) > 128:
            raise ValueError("the reordering takes at most 128 layers")
        self.stack, self.beams, self.groups, self.rows = stack, beams, groups, rows
        self.max_new, self.eos, self.page_size = max_new, eos, page_size
        columns = -(-stack.max_seq // page_size)
        # a request's prompt once and, per beam, the pages of max_new tokens and the unfilled one
        self.n_pages = groups * (columns + beams * (-(-max_new // page_size) + 1))
        if self.n_pages * page_size * dims.n_kv_heads >= 1 << 31:
            raise ValueError("the search needs more cache rows than pages can address")
        shape = (self.n_pages, dims.n_kv_heads, page_size, dims.head_dim)
        self.caches = PagedCacheList([PagedCache(torch.zeros(shape, dtype=dt, device=dev),
                                                 torch.zeros(shape, dtype=dt, device=dev)) for _ in stack.blocks])

        def i32(*size):
            return torch.zeros(size, dtype=torch.int32, device=dev)

        self.free = torch.arange(self.n_pages, dtype=torch.int32, device=dev)
        self.pool = torch.tensor([self.n_pages, 0], dtype=torch.int32, device=dev)
        self.table, self.home = i32(rows, columns), i32(rows, columns)   # home: the table as it was planned
        self.start, self.count, self.pos = i32(rows), i32(rows), i32(rows)
        self.err = i32(1)
        self.logits = torch.empty(rows, stack.vocab, dtype=torch.float32, device=dev)
        self.scores = torch.empty(rows, dtype=torch.float32, device=dev)
        self.parents, self.tokens, self.greedy = i32(rows), i32(rows), i32(rows)
        # a row per token, and one for the tokens of replays beyond max_new (sequences refuses them)
        self.all_parents, self.all_tokens = i32(max_new + 1, rows), i32(max_new + 1, rows)
        self.n = torch.zeros(1, dtype=torch.int64, device=dev)           # tokens chosen so far, on the device
        self.steps = 0                                                   # ... and on the host (begin and step calls)
        self.ws = torch.empty(stack.blocks[0].workspace_bytes(rows, 1), dtype=torch.uint8, device=dev)
        self.head_ws = torch.empty(llama_lmhead_workspace_bytes(rows, dims.d_model, stack.vocab), dtype=torch.uint8,
                                   device=dev)
        self.select_ws = torch.empty(llama_beam_select_workspace_bytes(groups, beams, stack.vocab, beams),
                                     dtype=torch.uint8, device=dev)
        self.act = [torch.empty(rows, 1, dims.d_model, dtype=dt, device=dev) for _ in range(2)]
        self.active = False
        # the calls may go to other streams than the one that filled all this
        torch.cuda.current_stream(dev).synchronize()

    def _choose(self, last, stream) -> None:
        # the best continuations; the states of the beams follow
        llama_beam_select(self.logits, self.scores, self.beams, self.beams, self.parents, self.tokens, self.scores,
                          self.select_ws, last=last, eos=self.eos, stream=stream)
        with LlamaStack._on(stream):
            at = self.n.clamp(max=self.max_new)
            self.all_parents.index_copy_(0, at, self.parents[None])
            self.all_tokens.index_copy_(0, at, self.tokens[None])
            self.n.add_(1)
        llama_beam_reorder(self.parents, self.beams, self.pos, self.table, self.caches, err_dev=self.err, stream=stream)

    def begin(self, ids: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
        """ids [requests, T] int32 on the device: prefill, pages for the prompts and max_new tokens, and the first
        token of every beam."""
        if self.active:
            raise RuntimeError("end() the running search first")
        st, ps, K = self.stack, self.page_size, self.beams
        if ids.dim() != 2 or ids.shape[0] != self.groups or ids.dtype != torch.int32:
            raise ValueError(f"ids must be int32 [{self.groups}, T]")
        T = ids.shape[1]
        if not 1 <= T <= st.prefill_tokens or T + self.max_new > st.max_seq:
            raise ValueError("the prompt must fit the stack's prefill, and with max_new its max_seq")
        st.prefill(ids, stream)
        with LlamaStack._on(stream):
            # beam 0 of a request holds the whole prompt, the others its unfilled page on
            full = T // ps * ps
            first = torch.arange(self.rows, device=ids.device) % K == 0
            self.start.copy_(torch.where(first, 0, full))
            self.count.copy_(torch.where(first, T + self.max_new, T - full + self.max_new))
            self.pos.fill_(T)
            self.table.fill_(-1)   # no page: a step beyond what is planned writes none
            slots = torch.empty(self.rows, T + self.max_new, dtype=torch.int32, device=ids.device)
        llama_paged_plan(self.start, self.count, ps, self.n_pages, self.free, self.pool, self.table, slots,
                         err_dev=self.err, stream=stream)
        with LlamaStack._on(stream):
            self.home.copy_(self.table)
            prompt_slots = slots.view(self.groups, K, -1)[:, 0, :T].contiguous()
        for cache, paged in zip(st.caches, self.caches.caches):
            llama_paged_store(cache.k, cache.v, prompt_slots, paged, err_dev=self.err, stream=stream)
        with LlamaStack._on(stream):
            self.logits.view(self.groups, K, -1)[:, 0].copy_(st.logits)   # the other rows are not read
            self.scores.copy_(torch.where(first, 0.0, float("-inf")))
            self.n.zero_()
            slots.record_stream(torch.cuda.current_stream())
            prompt_slots.record_stream(torch.cuda.current_stream())
        self.steps = 1
        self.active = True
        self._choose(None, stream)

    def step(self, stream: Optional[torch.cuda.Stream] = None) -> None:
        """One more token for every beam.  Reads nothing on the host: a captured graph of it can be replayed, as
        long as replays and calls together stay below max_new tokens."""
        if not self.active:
            raise RuntimeError("begin() first")
        if self.steps >= self.max_new:
            raise RuntimeError("max_new tokens were chosen")
        st = self.stack
        x, y = self.act
        llama_embed(self.tokens, self.rows, st.w_embed, st.vocab, st.dims.d_model, x, self.err, stream)
        for blk, cache in zip(st.blocks, self.caches.caches):
            blk.decode_paged(x, cache, self.table, self.pos, y, self.ws, stream)
            x, y = y, x
        llama_lmhead_argmax(x, self.rows, st.dims.d_model, st.g_final, st.w_out, st.vocab, st.dims.d_model, st.dims.eps,
                            self.greedy, self.logits, self.head_ws, self.head_ws.numel(), stream)
        with LlamaStack._on(stream):
            self.pos.add_(1)
        self.steps += 1
        self._choose(self.tokens if self.eos >= 0 else None, stream)

    def sequences(self):
        """(tokens [requests, beams, chosen], scores [requests, beams]), best first; waits for the device."""
        torch.cuda.synchronize(self.pos.device)      # the calls may have gone to any stream
        n = int(self.n.item())
        if n > self.max_new:
            raise RuntimeError("more than max_new tokens were chosen")
        row = torch.arange(self.rows, device=self.pos.device)
        out = torch.empty(self.rows, n, dtype=torch.int32, device=self.pos.device)
        for t in range(n - 1, -1, -1):
            out[:, t] = self.all_tokens[t][row]
            row = self.all_parents[t][row].long()
        scores = self.scores.view(self.groups, self.beams).clone()
        torch.cuda.synchronize(self.pos.device)      # read before a next call on another stream writes
        return out.view(self.groups, self.beams, n), scores

    def end(self, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Give the pages back."""
        if self.active:
            llama_paged_release(self.start, self.count, self.page_size, self.n_pages, self.free, self.pool, self.home,
                                err_dev=self.err, stream=stream)
            self.active = False

    def poll_error(self) -> int:
        """The first code on record: of the blocks, of the prompt's ids, of the search's own calls.  A code is
        cleared when it is returned, and not before."""
        torch.cuda.synchronize(self.pos.device)
        rc = self.stack.poll_error()
        for word in (self.stack.err, self.err):
            if rc == 0:
                rc = int(word.item())
                if rc:
                    word.zero_()
                    torch.cuda.synchronize(self.pos.device)
        return rc
