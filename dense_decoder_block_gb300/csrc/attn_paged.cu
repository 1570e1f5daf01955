// llama_paged_attention: one new token per sequence over a paged KV cache.
//
// The kernels are the decode attention of the block with the rows found through a
// block table (attn_simt.cu, attn_tc.cu): 128-key chunks spread over the SMs, each
// leaving (m, l, o), and a combine that folds a row's chunks in ascending order -- so
// the result does not depend on the batch, on the pages or on the split.
#include <algorithm>

#include "internal.h"

using namespace llama;

namespace {

bool heads_ok(int n_heads, int n_kv_heads, int head_dim) {
    return n_heads > 0 && n_kv_heads > 0 && n_heads <= 65535 && n_heads % n_kv_heads == 0 &&
           n_heads / n_kv_heads <= 64 && (head_dim == 32 || head_dim == 64 || head_dim == 128);
}
int chunks_of(int max_len) { return (int)(((long long)max_len + kAttnChunk - 1) / kAttnChunk); }

}  // namespace

extern "C" size_t llama_paged_attention_workspace_bytes(int batch, int n_heads, int n_kv_heads, int head_dim,
                                                        int max_len) {
    if (batch <= 0 || max_len <= 0 || !heads_ok(n_heads, n_kv_heads, head_dim)) return 0;
    return attn_decode_partial_bytes(batch, n_kv_heads, chunks_of(max_len), n_heads / n_kv_heads, head_dim);
}

extern "C" int llama_paged_attention(const void* q, int batch, int n_heads, int n_kv_heads, int head_dim, int dtype,
                                     const llama_paged_cache* kv, const int32_t* table, int table_stride,
                                     const int32_t* lens, int max_len, void* o, void* ws, size_t ws_bytes,
                                     int32_t* err_dev, void* stream) {
    if (batch < 0 || batch > 65535 || max_len <= 0 || table_stride <= 0) return LLAMA_ERR_INVALID_ARG;
    if (!heads_ok(n_heads, n_kv_heads, head_dim)) return LLAMA_ERR_UNSUPPORTED_DIMS;
    const int rc = paged_cache_check(kv, n_kv_heads, head_dim, dtype);
    if (rc != LLAMA_OK) return rc;
    if (batch == 0) return LLAMA_OK;
    // the kernels count (sequence, KV head, chunk) units of up to 1024 sequences, 8 query heads
    // each, in 32 bits
    if ((long long)std::min(batch, 1024) * n_heads * chunks_of(max_len) > INT32_MAX) return LLAMA_ERR_UNSUPPORTED_DIMS;
    if (!q || !o || !table || !lens || ((uintptr_t)q & 15) || ((uintptr_t)o & 15)) return LLAMA_ERR_INVALID_ARG;
    if (!ws || ws_bytes < llama_paged_attention_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, max_len))
        return LLAMA_ERR_WORKSPACE;
    if ((uintptr_t)ws & 15) return LLAMA_ERR_INVALID_ARG;
    AttnArgs a;
    a.q = q;
    a.o = o;
    a.kc = kv->k;
    a.vc = kv->v;
    a.batch = batch;
    a.tokens = 1;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.kv_seq = kv->page_size;
    a.pos_seq = lens;
    a.pos_off = -1;
    a.pages.table = table;
    a.pages.stride = table_stride;
    a.pages.n_pages = kv->n_pages;
    a.pages.shift = page_shift(kv->page_size);
    // positions must fit max_len and the table row
    const long long room = (long long)table_stride * kv->page_size;
    a.max_pos = room < max_len ? (int)room : max_len;
    a.dtype = dtype;
    a.partial = (float*)ws;
    a.n_chunks = chunks_of(max_len);
    a.err = err_dev;
    return launch_attention_paged(a, (cudaStream_t)stream) == cudaSuccess ? LLAMA_OK : LLAMA_ERR_CUDA;
}
