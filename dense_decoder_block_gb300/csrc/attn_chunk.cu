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

bool heads_ok(int n_heads, int n_kv_heads, int head_dim) {
    return n_heads > 0 && n_kv_heads > 0 && n_heads <= 65535 && n_heads % n_kv_heads == 0 &&
           n_heads / n_kv_heads <= 64 && (head_dim == 32 || head_dim == 64 || head_dim == 128);
}

// CTAs among which tiles may be split: ChunkWalk's rule at the most tiles and work of a launch (its fp32 arithmetic is
// within a thousandth); whole tiles go to no more.  All of them where no tile is ever cut: nothing is left in the workspace
// then.
int split_ctas(const ChunkDeal& d, int batch, int tokens, int n_kv_heads, int max_pos) {
    if (max_pos < kNeverSplit) return d.ctas;
    const double tiles = (double)std::min(batch, d.seqs) * n_kv_heads * ((tokens - 1) / d.tq + 1);
    const double work = tiles * ((double)max_pos + kTileKeys);
    const double n = std::min(work / d.min_stretch, d.pieces * std::sqrt(work * tiles / kAttnChunk));
    return (int)std::min((double)d.ctas, std::max(tiles, 1.001 * n + 1));
}

// rows of partials (m, l, o): two of a tile's rows for each of these CTAs
size_t partial_rows(const ChunkDeal& d, int split, int max_pos) {
    return max_pos < kNeverSplit ? 0 : (size_t)2 * split * d.rows;
}
// rows of O carried over: a tile's for each of them
size_t carry_rows(const ChunkDeal& d, int split, int max_pos) {
    return max_pos <= d.carry_keys ? 0 : (size_t)split * d.rows;
}

}  // namespace

// the partials, what is carried over, and where the CTAs begin
size_t attn_chunk_workspace_bytes(int dtype, int batch, int tokens, int n_heads, int n_kv_heads, int head_dim, int max_pos) {
    const int n_rep = n_heads / n_kv_heads;
    const ChunkDeal d = dtype == LLAMA_BF16 ? chunk_deal_tc(n_rep) : chunk_deal_f32(n_rep, head_dim);
    const int split = split_ctas(d, batch, tokens, n_kv_heads, max_pos);
    return (partial_rows(d, split, max_pos) * (head_dim + 2) + carry_rows(d, split, max_pos) * head_dim) * sizeof(float) +
           kChunkMaxCtas * (sizeof(int4) + sizeof(int));
}

int attn_chunk_launches(const AttnArgs& a) {
    return (a.batch + kTcSeqs - 1) / kTcSeqs * (device_sm_count() == 1 || a.max_pos < kNeverSplit ? 1 : 2);
}

cudaError_t launch_attention_chunk(const AttnArgs& a, const int* start, const int* count, void* ws, cudaStream_t s) {
    ChunkArgs k{};
    k.q = a.q;
    k.o = a.o;
    k.kc = a.kc;
    k.vc = a.vc;
    k.batch = a.batch;
    k.tokens = a.tokens;
    k.n_heads = a.n_heads;
    k.n_kv_heads = a.n_kv_heads;
    k.max_pos = a.max_pos;
    k.start = start;
    k.count = count;
    k.pages = a.pages;
    k.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)a.head_dim));
    const int n_rep = a.n_heads / a.n_kv_heads;
    const ChunkDeal d = a.dtype == LLAMA_BF16 ? chunk_deal_tc(n_rep) : chunk_deal_f32(n_rep, a.head_dim);
    k.tq = d.tq;
    k.join_keys = d.join_keys;
    k.min_stretch = d.min_stretch;
    k.pieces = d.pieces;
    k.split_ctas = split_ctas(d, a.batch, a.tokens, a.n_kv_heads, a.max_pos);
    const size_t rows = partial_rows(d, k.split_ctas, a.max_pos);
    k.partial = (float*)ws;
    k.part_ml = (float2*)(k.partial + rows * a.head_dim);
    k.carry = (float*)(k.part_ml + rows);
    k.cuts = (int4*)(k.carry + carry_rows(d, k.split_ctas, a.max_pos) * a.head_dim);
    k.cut_tokens = (int*)(k.cuts + kChunkMaxCtas);
    k.err = a.err;
    return a.dtype == LLAMA_BF16 ? launch_chunk_tc(k, a.head_dim, s) : launch_chunk_f32(k, a.head_dim, s);
}

}  // namespace llama

using namespace llama;

extern "C" size_t llama_paged_chunk_attention_workspace_bytes(int batch, int tokens, int n_heads, int n_kv_heads,
                                                              int head_dim, int max_len) {
    if (batch <= 0 || batch > 65535 || tokens <= 0 || (long long)batch * tokens > INT32_MAX || max_len <= 0 ||
        !heads_ok(n_heads, n_kv_heads, head_dim))
        return 0;   // as the call refuses
    // heads of 128 are of either type
    const size_t f32 = attn_chunk_workspace_bytes(LLAMA_F32, batch, tokens, n_heads, n_kv_heads, head_dim, max_len);
    if (head_dim != 128) return f32;
    return std::max(f32, attn_chunk_workspace_bytes(LLAMA_BF16, batch, tokens, n_heads, n_kv_heads, head_dim, max_len));
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
    AttnArgs a;
    a.q = q;
    a.o = o;
    a.kc = kv->k;
    a.vc = kv->v;
    a.batch = batch;
    a.tokens = tokens;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.pages.table = table;
    a.pages.stride = table_stride;
    a.pages.n_pages = kv->n_pages;
    a.pages.shift = page_shift(kv->page_size);
    // positions must fit max_len, the table row and 2^30 (sums of two of them fit an int)
    const long long room = std::min((long long)table_stride * kv->page_size, 1LL << 30);
    a.max_pos = room < max_len ? (int)room : max_len;
    a.dtype = dtype;
    a.err = err_dev;
    const cudaError_t e = launch_attention_chunk(a, start, count, ws, (cudaStream_t)stream);
    return e == cudaSuccess ? LLAMA_OK : LLAMA_ERR_CUDA;
}
