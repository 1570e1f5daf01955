// llama_paged_chunk_attention: a chunk of new tokens per sequence over a paged KV cache.
//
// "Llama 3.1 70B", Grouped-Query Attention, with the rows found through a block table: token t of
// sequence b attends positions 0 .. start[b] + t.
#include <algorithm>
#include <cmath>

#include "attn_chunk.cuh"
#include "internal.h"

namespace llama {
namespace {

__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ void from_f(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f(float* p, float v) { *p = v; }

// New tokens of sequence b: 0 (recorded) where its words are out of range.
__device__ __forceinline__ int chunk_count(const ChunkArgs& a, int b, int& start) {
    start = a.start[b];
    const int count = a.count[b];
    if (start >= 0 && count >= 0 && count <= a.tokens && (long long)start + count <= a.max_pos) return count;
    record_error(a.err, LLAMA_ERR_POS_RANGE);
    return 0;
}

// A warp per query row, its lanes sharing the row's columns, one key after another.
template <typename T, int DH>
__global__ void __launch_bounds__(256) k_attn_chunk_rows(const ChunkArgs a) {
    constexpr int DPL = DH / 32;
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t = (int)(w / a.n_heads), h = (int)(w % a.n_heads);
    int start;
    const int count = chunk_count(a, b, start);
    if (t >= count) return;
    const int g = h / (a.n_heads / a.n_kv_heads);
    const size_t row = ((size_t)b * a.tokens + t) * a.n_heads + h;
    float q[DPL], o[DPL], m = -INFINITY, l = 0.f;
    for (int e = 0; e < DPL; ++e) {
        q[e] = to_f(static_cast<const T*>(a.q)[row * DH + lane * DPL + e]);
        o[e] = 0.f;
    }
    const int shift = a.pages.shift;
    size_t base = 0;
    for (int j = 0; j <= start + t; ++j) {
        if ((j & ((1 << shift) - 1)) == 0)
            base = (((size_t)max(page_of(a.pages, b, j >> shift, a.err), 0) * a.n_kv_heads + g) << shift) * DH;
        const size_t at = base + (size_t)(j & ((1 << shift) - 1)) * DH + lane * DPL;
        float s = 0.f;
        for (int e = 0; e < DPL; ++e) s = fmaf(q[e], to_f(static_cast<const T*>(a.kc)[at + e]), s);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.scale_log2;
        const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
        const float c = exp2f(m - ref), p = exp2f(s - ref);
        l = fmaf(l, c, p);
        for (int e = 0; e < DPL; ++e) o[e] = fmaf(o[e], c, p * to_f(static_cast<const T*>(a.vc)[at + e]));
        m = mn;
    }
    for (int e = 0; e < DPL; ++e) from_f(static_cast<T*>(a.o) + row * DH + lane * DPL + e, o[e] / l);
}

template <typename T, int DH>
cudaError_t launch_rows(const ChunkArgs& a, cudaStream_t s) {
    const long long ctas = ((long long)a.tokens * a.n_heads + 7) / 8;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl(k_attn_chunk_rows<T, DH>, dim3((unsigned)ctas, a.batch), dim3(256), 0, s, a);
}

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
    cudaError_t e;
    if (dtype == LLAMA_BF16) e = launch_chunk_tc(a, head_dim, s);
    else if (head_dim == 32) e = launch_rows<float, 32>(a, s);
    else if (head_dim == 64) e = launch_rows<float, 64>(a, s);
    else e = launch_rows<float, 128>(a, s);
    return e == cudaSuccess ? LLAMA_OK : LLAMA_ERR_CUDA;
}
