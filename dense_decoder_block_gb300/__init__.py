"""GB300 (sm_103a) Llama-3-style decoder block: Python binding of libllama_block.so.

The functions here keep the C ABI's names and only marshal arguments (torch
tensors -> device pointers, the current CUDA stream -> cudaStream_t); every
step of the block runs in the library's CUDA kernels.  There is no fallback:
importing works without the library, but every call raises if it is missing.

    blk = LlamaBlock(dims, weights)            # weights: dict of CUDA tensors
    ws = blk.workspace(batch, tokens)
    blk.prefill(x, kv, y, ws)                  # x, y [B, T, d]
    blk.decode(x, kv, pos, y, ws)              # x, y [B, 1, d]
"""
from __future__ import annotations

import ctypes as C
from typing import Dict, Optional

import torch

from . import _native
from ._native import (LLAMA_BF16, LLAMA_F32, LLAMA_OK, LLAMA_ERR_INVALID_ARG, LLAMA_ERR_UNSUPPORTED_DIMS,
                      LLAMA_ERR_POS_RANGE, LLAMA_ERR_WORKSPACE, LLAMA_ERR_CUDA, LLAMA_ERR_DEVICE_TIMEOUT,
                      LLAMA_ERR_NO_PAGES, llama_block_dims, llama_block_weights, llama_kv_cache, llama_paged_cache,
                      llama_rope_scaling)

_raw_stream = torch._C._cuda_getCurrentRawStream

__all__ = [
    "LlamaBlock", "LlamaError", "KVCache", "lib", "llama_block_create", "llama_block_create_scaled",
    "llama_block_destroy",
    "llama_block_workspace_bytes", "llama_block_workspace_offsets", "llama_block_prefill", "llama_block_prefill_at", "llama_block_decode",
    "llama_block_decode_devpos", "llama_block_decode_seqpos",
    "llama_block_poll_error", "llama_block_last_error", "llama_block_selftest_wait_timeout", "Trace", "llama_block_set_stage_events", "llama_block_launch_count", "HostMapped",
    "llama_embed", "llama_lmhead_workspace_bytes",
    "llama_lmhead_argmax", "llama_lmhead_argmax_noalloc", "llama_sample", "llama_rmsnorm", "LLAMA_BF16", "LLAMA_F32",
    "PagedCache", "PagedCacheList", "llama_paged_plan", "llama_paged_release", "llama_paged_store",
    "llama_paged_attention", "llama_paged_attention_workspace_bytes", "llama_block_decode_paged",
    "llama_beam_select", "llama_beam_select_workspace_bytes", "llama_beam_reorder",
]


class LlamaError(RuntimeError):
    def __init__(self, code: int, msg: str = ""):
        self.code = code
        super().__init__(f"{_native.ERROR_NAMES.get(code, code)}: {msg}")


def lib():
    return _native.load()


class HostMapped:
    """A pinned host tensor seen through its device address: passed as x or y of
    prefill/decode, the kernels read or write the host memory directly."""

    def __init__(self, t: torch.Tensor):
        if t.is_cuda or not t.is_pinned():
            raise ValueError("HostMapped needs a pinned host tensor")
        if not t.is_contiguous():
            raise ValueError("HostMapped needs a contiguous tensor")
        dev = C.c_void_p()
        rc = lib().llama_device_ptr_of_host(C.c_void_p(t.data_ptr()), C.byref(dev))
        if rc != LLAMA_OK or not dev.value:
            raise LlamaError(rc, "llama_device_ptr_of_host: not pinned and mapped")
        self.t = t
        self.dev_ptr = dev.value
        self.shape = t.shape


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, HostMapped):
        return C.c_void_p(t.dev_ptr)
    if not t.is_cuda:
        raise ValueError("tensors passed to the block library must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the block library must be contiguous")
    return C.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream] = None):
    # the raw handle of the current stream: a torch.cuda.Stream object would take longer
    # to build (3 us) than a launch
    return stream.cuda_stream if stream is not None else _raw_stream(torch.cuda.current_device())


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return LLAMA_BF16
    if dt == torch.float32:
        return LLAMA_F32
    raise ValueError(f"unsupported dtype {dt}")


# ----------------------------------------------------------------------------- same-named wrappers

def llama_block_create(dims: llama_block_dims, weights: llama_block_weights) -> C.c_void_p:
    h = C.c_void_p()
    rc = lib().llama_block_create(C.byref(dims), C.byref(weights), C.byref(h))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_block_create")
    return h


def llama_block_create_scaled(dims: llama_block_dims, weights: llama_block_weights,
                              scaling: Optional[llama_rope_scaling]) -> C.c_void_p:
    h = C.c_void_p()
    rc = lib().llama_block_create_scaled(C.byref(dims), C.byref(weights),
                                         C.byref(scaling) if scaling is not None else None, C.byref(h))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_block_create_scaled")
    return h


def llama_block_destroy(h) -> None:
    lib().llama_block_destroy(h)


def llama_block_workspace_bytes(h, batch: int, tokens: int) -> int:
    return int(lib().llama_block_workspace_bytes(h, batch, tokens))


INTERMEDIATES = ("xn", "q", "o", "h", "hn", "u")


def llama_block_workspace_offsets(h, batch: int, tokens: int):
    """Byte offsets in the workspace of xn, q, o, h, hn, u for a call of this shape."""
    arr = (C.c_size_t * _native.LLAMA_BLOCK_INTERMEDIATES)()
    rc = lib().llama_block_workspace_offsets(h, batch, tokens, arr, _native.LLAMA_BLOCK_INTERMEDIATES)
    if rc != _native.LLAMA_BLOCK_INTERMEDIATES:
        raise LlamaError(rc, "llama_block_workspace_offsets")
    return dict(zip(INTERMEDIATES, (int(v) for v in arr)))


def llama_block_last_error(h) -> str:
    r = lib().llama_block_last_error(h)
    return r.decode() if r else ""


def _check(h, rc, what):
    if rc != LLAMA_OK:
        raise LlamaError(rc, f"{what}: {llama_block_last_error(h)}")


def llama_block_prefill(h, x, batch, tokens, kv: llama_kv_cache, y, ws, ws_bytes, stream=None) -> None:
    _check(h, lib().llama_block_prefill(h, _ptr(x), batch, tokens, C.byref(kv), _ptr(y), _ptr(ws), ws_bytes,
                                        _stream(stream)), "llama_block_prefill")


def llama_block_prefill_at(h, x, batch, tokens, start_pos, kv: llama_kv_cache, y, ws, ws_bytes, stream=None) -> None:
    _check(h, lib().llama_block_prefill_at(h, _ptr(x), batch, tokens, start_pos, C.byref(kv), _ptr(y), _ptr(ws),
                                           ws_bytes, _stream(stream)), "llama_block_prefill_at")


def llama_block_decode(h, x, batch, kv: llama_kv_cache, pos, y, ws, ws_bytes, stream=None) -> None:
    _check(h, lib().llama_block_decode(h, _ptr(x), batch, C.byref(kv), int(pos), _ptr(y), _ptr(ws), ws_bytes,
                                       _stream(stream)), "llama_block_decode")


def llama_block_decode_devpos(h, x, batch, kv: llama_kv_cache, pos_dev, y, ws, ws_bytes, stream=None) -> None:
    _check(h, lib().llama_block_decode_devpos(h, _ptr(x), batch, C.byref(kv), _ptr(pos_dev), _ptr(y), _ptr(ws),
                                              ws_bytes, _stream(stream)), "llama_block_decode_devpos")


def llama_block_decode_seqpos(h, x, batch, kv: llama_kv_cache, pos_seq, y, ws, ws_bytes, stream=None) -> None:
    _check(h, lib().llama_block_decode_seqpos(h, _ptr(x), batch, C.byref(kv), _ptr(pos_seq), _ptr(y), _ptr(ws),
                                              ws_bytes, _stream(stream)), "llama_block_decode_seqpos")


def llama_block_decode_paged(h, x, batch, kv: llama_paged_cache, table, pos_seq, y, ws, ws_bytes, stream=None) -> None:
    _check(h, lib().llama_block_decode_paged(h, _ptr(x), batch, C.byref(kv), _ptr(table), table.shape[1], _ptr(pos_seq),
                                             _ptr(y), _ptr(ws), ws_bytes, _stream(stream)), "llama_block_decode_paged")


def llama_block_set_stage_events(h, events) -> None:
    """events: None, or a list of LLAMA_BLOCK_STAGES + 1 torch.cuda.Event (enable_timing=True)."""
    if events is None:
        rc = lib().llama_block_set_stage_events(h, None, 0)
    else:
        arr = (C.c_void_p * len(events))(*[C.c_void_p(e.cuda_event) for e in events])
        rc = lib().llama_block_set_stage_events(h, arr, len(events))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_block_set_stage_events")


def llama_block_launch_count(h) -> int:
    """Kernels enqueued by the last successful prefill/decode call on the handle."""
    return int(lib().llama_block_launch_count(h))


def llama_block_poll_error(h, stream=None) -> int:
    return int(lib().llama_block_poll_error(h, _stream(stream)))


class Trace:
    """Per-CTA timeline of the block's kernels while the context is open
    (llama_trace_begin / llama_trace_end; the trace build of the library only:
    load it with `_native.load(build.build(trace=True))` before the first call).
    After exit, `records()` gives the columns kernel, sm, cta, t_start,
    t_release, t_end (ns) on the host."""

    def __init__(self, capacity: int = 1 << 16, device=None):
        import torch
        dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.capacity = int(capacity)
        self.buf = torch.zeros(self.capacity, 4, dtype=torch.int64, device=dev)
        self.count = torch.zeros(1, dtype=torch.int32, device=dev)

    def __enter__(self):
        rc = lib().llama_trace_begin(_ptr(self.buf), _ptr(self.count), self.capacity)
        if rc != LLAMA_OK:
            raise LlamaError(rc, "llama_trace_begin")
        return self

    def __exit__(self, *exc):
        lib().llama_trace_end()
        return False

    def records(self):
        import torch
        torch.cuda.synchronize(self.buf.device)
        n = min(int(self.count.item()), self.capacity)
        r = self.buf[:n].cpu()
        w0 = r[:, 0]
        return {"kernel": (w0 & 0xffff).tolist(), "sm": ((w0 >> 16) & 0xffff).tolist(),
                "cta": ((w0 >> 32) & 0xffffffff).tolist(), "t_start": r[:, 1].tolist(),
                "t_release": r[:, 2].tolist(), "t_end": r[:, 3].tolist(), "claimed": int(self.count.item())}


def llama_block_selftest_wait_timeout(h, budget_ns, stream=None) -> None:
    _check(h, lib().llama_block_selftest_wait_timeout(h, int(budget_ns), _stream(stream)),
           "llama_block_selftest_wait_timeout")


def llama_rmsnorm(x, g, y, rows, d, eps, stream=None) -> None:
    rc = lib().llama_rmsnorm(_ptr(x), _ptr(g), _ptr(y), rows, d, C.c_float(eps), _dtype_code(x.dtype),
                             _stream(stream))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_rmsnorm")


def llama_embed(ids, n_tokens, w_embed, vocab, d_model, x, err_dev=None, stream=None) -> None:
    rc = lib().llama_embed(_ptr(ids), n_tokens, _ptr(w_embed), vocab, d_model, _ptr(x), _ptr(err_dev),
                           _stream(stream))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_embed")


def llama_lmhead_workspace_bytes(batch, d_model, vocab) -> int:
    return int(lib().llama_lmhead_workspace_bytes(batch, d_model, vocab))


def llama_lmhead_argmax(h, batch, h_stride, g_final, w_out, vocab, d_model, eps, ids, logits, ws, ws_bytes,
                        stream=None) -> None:
    rc = lib().llama_lmhead_argmax(_ptr(h), batch, h_stride, _ptr(g_final), _ptr(w_out), vocab, d_model,
                                   C.c_float(eps), _ptr(ids), _ptr(logits), _ptr(ws), ws_bytes, _stream(stream))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_lmhead_argmax")


def llama_lmhead_argmax_noalloc(h, batch, h_stride, g_final, w_out, vocab, d_model, eps, ids, logits,
                                stream=None) -> None:
    """The LM head + greedy choice without a workspace (library-owned scratch; see the header)."""
    rc = lib().llama_lmhead_argmax_noalloc(_ptr(h), batch, h_stride, _ptr(g_final), _ptr(w_out), vocab, d_model,
                                           C.c_float(eps), _ptr(ids), _ptr(logits), _stream(stream))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_lmhead_argmax_noalloc")


def llama_sample(logits, batch, vocab, temperature, top_k, top_p, uniforms, ids, stream=None) -> None:
    """ids[b] drawn from softmax(logits[b] / temperature) after top-k / top-p, with uniforms[b]."""
    rc = lib().llama_sample(_ptr(logits), batch, vocab, C.c_float(temperature), int(top_k), C.c_float(top_p),
                            _ptr(uniforms), _ptr(ids), _stream(stream))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_sample")


# ----------------------------------------------------------------------------- paged cache and beam search

def _arg(t, name: str, dtype: torch.dtype, least: int, device=None):
    """The address of a contiguous CUDA tensor of `dtype` with at least `least` elements
    on `device` (default: the current one)."""
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {dtype} expected, got {t.dtype}")
    if t.get_device() != (torch.cuda.current_device() if device is None else device):   # -1 on the host
        raise ValueError(f"{name} must live on the current CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < least:
        raise ValueError(f"{name}: {least} elements needed, got {t.numel()}")
    return t.data_ptr()


def _err_arg(err_dev, device):
    return None if err_dev is None else _arg(err_dev, "err_dev", torch.int32, 1, device)


class PagedCache:
    """One layer's paged K and V: [n_pages, n_kv_heads, page_size, head_dim] each
    (caller-owned torch tensors)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if k.shape != v.shape or k.dim() != 4 or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must be alike: [n_pages, n_kv_heads, page_size, head_dim]")
        self.k, self.v = k, v
        self.dtype = k.dtype
        self.device = k.get_device() if k.is_cuda else -1
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.code = _dtype_code(k.dtype)
        self.c = llama_paged_cache(_ptr(k), _ptr(v), self.n_pages, self.page_size)
        self.ref = C.byref(self.c)


class PagedCacheList:
    """The caches of a stack's layers, addressed by one block table."""

    def __init__(self, caches):
        caches = list(caches)
        if not caches:
            raise ValueError("at least one layer")
        first = caches[0]
        if any(c.k.shape != first.k.shape or c.dtype != first.dtype or c.device != first.device for c in caches):
            raise ValueError("the layers' caches must be alike")
        if len({c.c.k for c in caches} | {c.c.v for c in caches}) != 2 * len(caches):
            raise ValueError("the layers' buffers must be distinct")
        self.caches, self.first = caches, first
        self.c = (llama_paged_cache * len(caches))(*[c.c for c in caches])

    def __len__(self):
        return len(self.caches)

    def __getitem__(self, i):
        return self.caches[i]


def _table_arg(table, name, rows, device):
    if table.dim() != 2 or table.shape[0] < rows:
        raise ValueError(f"{name} must be [{rows} rows or more, pages per row]")
    return _arg(table, name, torch.int32, 0, device)


def llama_paged_plan(start, count, page_size: int, n_pages: int, free_pages, pool, table, slots, pool_out=None,
                     err_dev=None, stream=None) -> None:
    """Block tables and slot maps: request b, holding start[b] positions, receives count[b] more; the pages
    they need come from the stack free_pages[: pool[0]].  slots [batch, tokens], table [batch, pages per row];
    pool_out defaults to pool (in place)."""
    dev = torch.cuda.current_device()
    batch = start.numel()
    if slots.dim() != 2 or slots.shape[0] != batch or count.numel() != batch:
        raise ValueError("start, count [batch] and slots [batch, tokens] must agree")
    out = pool if pool_out is None else pool_out
    rc = lib().llama_paged_plan(_arg(start, "start", torch.int32, batch, dev), _arg(count, "count", torch.int32, batch, dev),
                                batch, slots.shape[1], page_size, n_pages,
                                _arg(free_pages, "free_pages", torch.int32, n_pages, dev),
                                _arg(pool, "pool", torch.int32, 2, dev), _arg(out, "pool_out", torch.int32, 2, dev),
                                _table_arg(table, "table", batch, dev), table.shape[1],
                                _arg(slots, "slots", torch.int32, 0, dev), _err_arg(err_dev, dev), _stream(stream))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_paged_plan")


def llama_paged_release(start, count, page_size: int, n_pages: int, free_pages, pool, table, pool_out=None,
                        err_dev=None, stream=None) -> None:
    """The pages that a plan with the same start and count took go back on the stack."""
    dev = torch.cuda.current_device()
    batch = start.numel()
    if count.numel() != batch:
        raise ValueError("start and count [batch] must agree")
    out = pool if pool_out is None else pool_out
    rc = lib().llama_paged_release(_arg(start, "start", torch.int32, batch, dev),
                                   _arg(count, "count", torch.int32, batch, dev), batch, page_size, n_pages,
                                   _arg(free_pages, "free_pages", torch.int32, n_pages, dev),
                                   _arg(pool, "pool", torch.int32, 2, dev), _arg(out, "pool_out", torch.int32, 2, dev),
                                   _table_arg(table, "table", batch, dev), table.shape[1], _err_arg(err_dev, dev),
                                   _stream(stream))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_paged_release")


def llama_paged_store(k, v, slots, kv: PagedCache, src_pos: int = 0, err_dev=None, stream=None) -> None:
    """Rows src_pos + t of the contiguous k, v [batch, n_kv_heads, src_seq, head_dim] to the pages of kv, at
    slots [batch, tokens] (negative: skipped)."""
    dev = kv.device
    if k.dim() != 4 or k.shape != v.shape or k.shape[1] != kv.n_kv_heads or k.shape[3] != kv.head_dim:
        raise ValueError("k, v must be [batch, n_kv_heads, src_seq, head_dim] of the cache's heads")
    if slots.dim() != 2 or slots.shape[0] > k.shape[0]:
        raise ValueError("slots must be [batch, tokens]")
    _current(dev)
    rc = lib().llama_paged_store(_arg(k, "k", kv.dtype, 0, dev), _arg(v, "v", kv.dtype, 0, dev), slots.shape[0],
                                 slots.shape[1], k.shape[2], src_pos, _arg(slots, "slots", torch.int32, 0, dev),
                                 kv.n_kv_heads, kv.head_dim, kv.code, kv.ref, _err_arg(err_dev, dev), _stream(stream))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_paged_store")


def _current(device: int) -> None:
    if device != torch.cuda.current_device():
        raise ValueError("the cache's device is not the current device")


def llama_paged_attention_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, max_len) -> int:
    return int(lib().llama_paged_attention_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, max_len))


def llama_paged_attention(q, kv: PagedCache, table, lens, max_len: int, o, ws, err_dev=None, stream=None) -> None:
    """o[b] = attention of q[b] [n_heads, head_dim] over the first lens[b] positions of sequence b (0: zeros)."""
    dev = kv.device
    if q.dim() != 3 or q.shape[2] != kv.head_dim or o.shape != q.shape:
        raise ValueError("q and o must be [batch, n_heads, head_dim] of the cache's heads")
    batch, n_heads = q.shape[0], q.shape[1]
    _current(dev)
    rc = lib().llama_paged_attention(_arg(q, "q", kv.dtype, 0, dev), batch, n_heads, kv.n_kv_heads, kv.head_dim, kv.code,
                                     kv.ref, _table_arg(table, "table", batch, dev), table.shape[1],
                                     _arg(lens, "lens", torch.int32, batch, dev), max_len, _arg(o, "o", kv.dtype, 0, dev),
                                     _arg(ws, "ws", torch.uint8, 0, dev), ws.numel(), _err_arg(err_dev, dev),
                                     _stream(stream))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_paged_attention")


def llama_beam_select_workspace_bytes(groups, beams, vocab, n_out) -> int:
    return int(lib().llama_beam_select_workspace_bytes(groups, beams, vocab, n_out))


def llama_beam_select(logits, scores, beams: int, n_out: int, parents, tokens, out_scores, ws, last=None, eos: int = -1,
                      stream=None) -> None:
    """The n_out best continuations of each group of `beams` rows of logits [groups * beams, vocab] (fp32), given
    the rows' cumulative scores; rows whose last token is eos have ended.  Outputs [groups, n_out]."""
    dev = torch.cuda.current_device()
    if logits.dim() != 2 or beams < 1 or logits.shape[0] % beams:
        raise ValueError("logits must be [groups * beams, vocab]")
    rows, vocab = logits.shape
    groups = rows // beams
    n = groups * n_out
    rc = lib().llama_beam_select(_arg(logits, "logits", torch.float32, 0, dev), groups, beams, vocab,
                                 _arg(scores, "scores", torch.float32, rows, dev),
                                 None if last is None else _arg(last, "last", torch.int32, rows, dev), eos, n_out,
                                 _arg(parents, "parents", torch.int32, n, dev), _arg(tokens, "tokens", torch.int32, n, dev),
                                 _arg(out_scores, "out_scores", torch.float32, n, dev),
                                 _arg(ws, "ws", torch.uint8, 0, dev), ws.numel(), _stream(stream))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_beam_select")


def llama_beam_reorder(parents, beams: int, lens, table, caches: PagedCacheList, err_dev=None, stream=None) -> None:
    """Rows of table, and the unfilled last pages of every layer's cache, follow parents [groups * beams] in place."""
    f = caches.first
    dev = f.device
    rows = parents.numel()
    if beams < 1 or rows % beams:
        raise ValueError("parents must be [groups * beams]")
    _current(dev)
    rc = lib().llama_beam_reorder(_arg(parents, "parents", torch.int32, 0, dev), rows // beams, beams,
                                  _arg(lens, "lens", torch.int32, rows, dev), _table_arg(table, "table", rows, dev),
                                  table.shape[1], caches.c, len(caches), f.n_kv_heads, f.head_dim, f.code,
                                  _err_arg(err_dev, dev), _stream(stream))
    if rc != LLAMA_OK:
        raise LlamaError(rc, "llama_beam_reorder")


# ----------------------------------------------------------------------------- convenience

class KVCache:
    """K and V buffers [batch, n_kv_heads, max_seq, head_dim] (caller-owned torch tensors)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        assert k.shape == v.shape and k.dim() == 4
        self.k, self.v = k, v
        self.c = llama_kv_cache(C.c_void_p(k.data_ptr()), C.c_void_p(v.data_ptr()), k.shape[0], k.shape[2])


class LlamaBlock:
    """Owns a handle; borrows the weight tensors (kept referenced here)."""

    def __init__(self, dims, weights: Dict[str, torch.Tensor], gains: Dict[str, torch.Tensor], max_seq: int):
        dt = weights["wq"].dtype
        self.dims = dims
        self._keep = dict(weights, **gains)
        self.c_dims = llama_block_dims(dims.d_model, dims.n_heads, dims.n_kv_heads, dims.head_dim, dims.d_ff,
                                       max_seq, dims.eps, dims.rope_theta, _dtype_code(dt))
        names = ("g_attn", "wq", "wk", "wv", "wo", "g_ffn", "w_gate", "w_up", "w_down")
        self.c_w = llama_block_weights(*[_ptr(self._keep[n]) for n in names])
        sc = getattr(dims, "rope_scaling", None)   # (factor, low, high, original context) or None
        self.c_scaling = None if sc is None else llama_rope_scaling(float(sc[0]), float(sc[1]), float(sc[2]),
                                                                    int(sc[3]))
        self.h = llama_block_create_scaled(self.c_dims, self.c_w, self.c_scaling)

    def __del__(self):
        h = getattr(self, "h", None)
        if h is not None and _native._lib is not None:
            llama_block_destroy(h)
            self.h = None

    def workspace_bytes(self, batch: int, tokens: int) -> int:
        return llama_block_workspace_bytes(self.h, batch, tokens)

    def workspace(self, batch: int, tokens: int, device=None) -> torch.Tensor:
        n = self.workspace_bytes(batch, tokens)
        return torch.empty(n, dtype=torch.uint8, device=device or self._keep["wq"].device)

    def intermediates(self, ws: torch.Tensor, batch: int, tokens: int) -> Dict[str, torch.Tensor]:
        """Views of the workspace `ws` of a finished call (batch, tokens) as the block's
        intermediates xn, q, o, h, hn, u, each [batch * tokens, width]."""
        off = llama_block_workspace_offsets(self.h, batch, tokens)
        d = self.dims
        dt = self._keep["wq"].dtype
        es = torch.finfo(dt).bits // 8
        widths = {"xn": d.d_model, "q": d.q_dim, "o": d.q_dim, "h": d.d_model, "hn": d.d_model, "u": d.d_ff}
        M = batch * tokens
        out = {}
        for name, width in widths.items():
            nbytes = M * width * es
            out[name] = ws[off[name]:off[name] + nbytes].view(dt).view(M, width)
        return out

    def prefill(self, x, kv: KVCache, y, ws, stream=None):
        B, T = x.shape[0], x.shape[1]
        llama_block_prefill(self.h, x, B, T, kv.c, y, ws, ws.numel(), stream)

    def prefill_at(self, x, kv: KVCache, start_pos: int, y, ws, stream=None):
        """x [B, T, d] holds the tokens at positions start_pos .. start_pos + T - 1."""
        B, T = x.shape[0], x.shape[1]
        llama_block_prefill_at(self.h, x, B, T, start_pos, kv.c, y, ws, ws.numel(), stream)

    def decode(self, x, kv: KVCache, pos: int, y, ws, stream=None):
        llama_block_decode(self.h, x, x.shape[0], kv.c, pos, y, ws, ws.numel(), stream)

    def decode_devpos(self, x, kv: KVCache, pos_dev, y, ws, stream=None):
        llama_block_decode_devpos(self.h, x, x.shape[0], kv.c, pos_dev, y, ws, ws.numel(), stream)

    def decode_seqpos(self, x, kv: KVCache, pos_seq, y, ws, stream=None):
        """pos_seq: int32 CUDA tensor [batch], sequence b at position pos_seq[b]."""
        llama_block_decode_seqpos(self.h, x, x.shape[0], kv.c, pos_seq, y, ws, ws.numel(), stream)

    def decode_paged(self, x, kv: "PagedCache", table, pos_seq, y, ws, stream=None):
        """One step on a paged cache: sequence b at position pos_seq[b], its pages in row b of table
        [batch, pages per row] (int32 CUDA tensors)."""
        if kv.n_kv_heads != self.dims.n_kv_heads or kv.head_dim != self.dims.head_dim or \
                kv.dtype != self._keep["wq"].dtype:
            raise ValueError("the paged cache's heads or type are not the block's")
        _current(kv.device)
        _table_arg(table, "table", x.shape[0], None)
        _arg(pos_seq, "pos_seq", torch.int32, x.shape[0])
        llama_block_decode_paged(self.h, x, x.shape[0], kv.c, table, pos_seq, y, ws, ws.numel(), stream)

    def poll_error(self, stream=None) -> int:
        return llama_block_poll_error(self.h, stream)

    def selftest_wait_timeout(self, budget_ns, stream=None) -> None:
        llama_block_selftest_wait_timeout(self.h, budget_ns, stream)

    def launch_count(self) -> int:
        return llama_block_launch_count(self.h)
