// llama_paged_chunk_attention: a chunk of new tokens per sequence over a paged KV cache.
//
// "Llama 3.1 70B", Grouped-Query Attention, with the rows found through a block table: token t of
// sequence b attends positions 0 .. start[b] + t.  bf16 runs on the tensor cores (attn_chunk_tc.cu), fp32 on the CUDA
// cores (attn_chunk_f32.cu); both deal out the same tiles and chunks (attn_chunk.cuh).
#include <algorithm>
#include <cmath>

#include "attn_chunk.cuh"
#include "internal.h"

namespace llama {
namespace {

size_t align16(size_t v) { return (v + 15) & ~(size_t)15; }

bool heads_ok(int n_heads, int n_kv_heads, int head_dim) {
    return n_heads > 0 && n_kv_heads > 0 && n_heads <= 65535 && n_heads % n_kv_heads == 0 &&
           n_heads / n_kv_heads <= 64 && (head_dim == 32 || head_dim == 64 || head_dim == 128);
}

}  // namespace
}  // namespace llama

using namespace llama;

extern "C" size_t llama_paged_chunk_attention_workspace_bytes(int batch, int tokens, int n_heads, int n_kv_heads,
                                                              int head_dim, int max_len) {
    if (batch <= 0 || tokens <= 0 || max_len <= 0 || !heads_ok(n_heads, n_kv_heads, head_dim)) return 0;
    // two partials (m, l, o) of up to 256 rows for each CTA, and where the CTAs begin
    return align16((size_t)kChunkMaxCtas * 512 * (head_dim + 2) * sizeof(float)) + kChunkMaxCtas * sizeof(int4);
}

extern "C" int llama_paged_chunk_attention(const void* q, int batch, int tokens, int n_heads, int n_kv_heads,
                                           int head_dim, int dtype, const llama_paged_cache* kv, const int32_t* table,
                                           int table_stride, const int32_t* start, const int32_t* count, int max_len,
                                           void* o, void* ws, size_t ws_bytes, int32_t* err_dev, void* stream) {
    if (batch < 0 || batch > 65535 || tokens < 0 || max_len <= 0 || table_stride <= 0) return LLAMA_ERR_INVALID_ARG;
    if (!heads_ok(n_heads, n_kv_heads, head_dim)) return LLAMA_ERR_UNSUPPORTED_DIMS;
    const int rc = paged_cache_check(kv, n_kv_heads, head_dim, dtype);
    if (rc != LLAMA_OK) return rc;
    if ((long long)batch * tokens > INT32_MAX) return LLAMA_ERR_UNSUPPORTED_DIMS;
    if (batch == 0 || tokens == 0) return LLAMA_OK;
    if (!q || !o || !table || !start || !count || ((uintptr_t)q & 15) || ((uintptr_t)o & 15)) return LLAMA_ERR_INVALID_ARG;
    if (!ws || ws_bytes < llama_paged_chunk_attention_workspace_bytes(batch, tokens, n_heads, n_kv_heads, head_dim, max_len))
        return LLAMA_ERR_WORKSPACE;
    if ((uintptr_t)ws & 15) return LLAMA_ERR_INVALID_ARG;
    ChunkArgs a{};
    a.q = q;
    a.o = o;
    a.kc = kv->k;
    a.vc = kv->v;
    a.batch = batch;
    a.tokens = tokens;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.start = start;
    a.count = count;
    a.pages.table = table;
    a.pages.stride = table_stride;
    a.pages.n_pages = kv->n_pages;
    a.pages.shift = page_shift(kv->page_size);
    const long long room = (long long)table_stride * kv->page_size;
    a.max_pos = room < max_len ? (int)room : max_len;
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)head_dim));
    a.err = err_dev;
    a.partial = (float*)ws;
    a.part_ml = (float2*)(a.partial + (size_t)kChunkMaxCtas * 512 * head_dim);
    a.cuts = (int4*)((uint8_t*)ws + align16((size_t)kChunkMaxCtas * 512 * (head_dim + 2) * sizeof(float)));
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == LLAMA_BF16 ? launch_chunk_tc(a, head_dim, s) : launch_chunk_f32(a, head_dim, s);
    return e == cudaSuccess ? LLAMA_OK : LLAMA_ERR_CUDA;
}
