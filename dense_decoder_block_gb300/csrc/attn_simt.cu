// Causal GQA attention on CUDA cores, prefill and decode, with one shared
// reduction schedule.
//
// "Llama 3.1 70B", Grouped-Query Attention: scores q.k / sqrt(d_h), causal,
// softmax over keys, weights average V; query head h reads KV head
// h / (n_heads / n_kv_heads).  "Llama 3 8B · Prepare Q, K, V" (decode mode):
// K and V are cached at KV-head size and read once per group.
//
// Schedule.  Keys are cut into chunks of kAttnChunk = 128.  For one query row
// and one chunk a warp computes the chunk partial (m, l, o): m the chunk's max
// score (log2 domain), l = sum 2^(s - m), o = sum 2^(s - m) v.  Chunks are
// folded in ascending order from chunk 0.  The prefill kernel folds in
// registers as it walks the chunks; the decode kernel writes each chunk's
// partial to the workspace (split over CTAs) and the combine kernel folds them
// in the same order with the same function, so a decode row is bit-identical
// to the prefill row at the same position.  Keys past the query's position are
// neither scored nor loaded.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "attn_fold.cuh"
#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace llama {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRowsMax = 64;    // query rows per prefill CTA (n_rep * tokens)
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void ptx_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void ptx_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ void from_f(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f(float* p, float v) { *p = v; }

template <typename T, int DH>
struct Tile {
    static constexpr int VEC = 16 / sizeof(T);          // elements per 16-byte vector
    static constexpr int LD = DH + VEC;                  // padded row stride (elements)
    static constexpr int DPL = DH / 32;                  // output dims per lane
};

__device__ __forceinline__ void cp_async16(void* smem, const void* gmem, bool valid) {
    const unsigned s = (unsigned)__cvta_generic_to_shared(smem);
    const int src = valid ? 16 : 0;   // 0 -> zero fill, nothing read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(gmem), "r"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

// Load keys [key0, key0 + 128) of one (sequence, kv head) into smem; keys above
// last_key are zero-filled without touching global memory.
template <typename T, int DH>
__device__ __forceinline__ void load_chunk(T* Ks, T* Vs, const T* kc, const T* vc, size_t head_base, int key0,
                                           int last_key) {
    using TL = Tile<T, DH>;
    constexpr int VPR = DH / TL::VEC;   // vectors per row
    for (int v = threadIdx.x; v < kAttnChunk * VPR; v += kThreads) {
        const int j = v / VPR, c = (v % VPR) * TL::VEC;
        const int key = key0 + j;
        const bool ok = key <= last_key;
        const size_t g = head_base + (size_t)(ok ? key : 0) * DH + c;
        cp_async16(Ks + j * TL::LD + c, kc + g, ok);
        cp_async16(Vs + j * TL::LD + c, vc + g, ok);
    }
    cp_async_wait_all();
}

// q . k of one key (a row of the chunk)
template <typename T, int DH>
__device__ __forceinline__ float key_dot(const float* q, const T* kr) {
    constexpr int VEC = Tile<T, DH>::VEC;
    float acc = 0.f;
#pragma unroll 4
    for (int d = 0; d < DH; d += VEC) {
        T kv[VEC];
        *reinterpret_cast<uint4*>(kv) = *reinterpret_cast<const uint4*>(kr + d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc = __fmaf_rn(q[d + e], to_f(kv[e]), acc);
    }
    return acc;
}

// One warp: the weights of one query row (fp32 in smem) over one chunk, lane's keys
// lane + 32 i, with their maximum and sum.  jmax = last key index inside the chunk this
// row may see (0..127).
template <typename T, int DH>
__device__ __forceinline__ void chunk_weights(const float* q, const T* Ks, int jmax, float scale_log2, float& m_out,
                                              float& l_out, float (&p)[4]) {
    using TL = Tile<T, DH>;
    const int lane = threadIdx.x & 31;
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = lane + 32 * i;
        s[i] = j <= jmax ? __fmul_rn(key_dot<T, DH>(q, Ks + j * TL::LD), scale_log2) : -INFINITY;
    }
    float mx = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[i] = (lane + 32 * i <= jmax) ? exp2f(__fsub_rn(s[i], mx)) : 0.f;
        l = __fadd_rn(l, p[i]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l = __fadd_rn(l, __shfl_xor_sync(kFull, l, off));
    m_out = mx;
    l_out = __shfl_sync(kFull, l, 0);
}

// ... and the weights' average of V, not normalised: lane owns dims lane * DPL ...
template <typename T, int DH>
__device__ __forceinline__ void chunk_average(const T* Vs, int jmax, const float (&p)[4], float (&o)[DH / 32]) {
    using TL = Tile<T, DH>;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < TL::DPL; ++e) o[e] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (32 * i > jmax) break;
#pragma unroll 8
        for (int jj = 0; jj < 32; ++jj) {
            const int j = 32 * i + jj;
            if (j > jmax) break;
            const float pj = __shfl_sync(kFull, p[i], jj);
            const T* vr = Vs + j * TL::LD + lane * TL::DPL;
#pragma unroll
            for (int e = 0; e < TL::DPL; ++e) o[e] = __fmaf_rn(pj, to_f(vr[e]), o[e]);
        }
    }
}

// One warp: the partial of one query row over one chunk.
template <typename T, int DH>
__device__ __forceinline__ void chunk_partial(const float* q, const T* Ks, const T* Vs, int jmax, float scale_log2,
                                              float& m_out, float& l_out, float (&o)[DH / 32]) {
    float p[4];
    chunk_weights<T, DH>(q, Ks, jmax, scale_log2, m_out, l_out, p);
    chunk_average<T, DH>(Vs, jmax, p, o);
}

struct AttnK {
    const void* q;
    void* o;
    const void* kc;
    const void* vc;
    int batch, tokens, n_heads, n_kv_heads, kv_seq, start_pos, max_pos;
    const int* pos_dev;
    const int* pos_seq;   // decode combine: sequence b at position pos_seq[b]
    float scale_log2;
    float* partial;
    int n_chunks;
    int tq;    // prefill: tokens per CTA
    int* err;
};

__device__ __forceinline__ int base_position(const AttnK& a) { return a.pos_dev ? *a.pos_dev : a.start_pos; }

// ----------------------------------------------------------------------------- prefill
template <typename T, int DH>
__global__ void __launch_bounds__(kThreads) k_attn_prefill(const AttnK a) {
    using TL = Tile<T, DH>;
    constexpr int DPL = TL::DPL;
    constexpr int RPW = kRowsMax / kWarps;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    T* Ks = reinterpret_cast<T*>(smem_raw);
    T* Vs = Ks + kAttnChunk * TL::LD;
    float* qs = reinterpret_cast<float*>(Vs + kAttnChunk * TL::LD);

    ptx_wait();
    if (threadIdx.x == 0) ptx_launch_dependents();
    const int g = blockIdx.y, b = blockIdx.z;
    const int n_rep = a.n_heads / a.n_kv_heads;
    const int t0 = blockIdx.x * a.tq;
    const int rows = n_rep * a.tq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int base = base_position(a);
    const int t_last = min(t0 + a.tq, a.tokens) - 1;
    if (base < 0 || base + t_last >= a.max_pos) {
        if (threadIdx.x == 0) record_error(a.err, LLAMA_ERR_POS_RANGE);
        return;
    }
    const int pos_last = base + t_last;
    const T* q = reinterpret_cast<const T*>(a.q);
    const size_t qld = (size_t)a.n_heads * DH;
    for (int i = threadIdx.x; i < rows * DH; i += kThreads) {
        const int r = i / DH, d = i % DH;
        const int t = t0 + r / n_rep, h = g * n_rep + r % n_rep;
        qs[i] = (t < a.tokens) ? to_f(q[((size_t)b * a.tokens + t) * qld + (size_t)h * DH + d]) : 0.f;
    }
    float M[RPW], L[RPW], O[RPW][DPL];
    const size_t head_base = ((size_t)b * a.n_kv_heads + g) * a.kv_seq * DH;
    const int n_chunks = pos_last / kAttnChunk + 1;
    for (int c = 0; c < n_chunks; ++c) {
        __syncthreads();
        load_chunk<T, DH>(Ks, Vs, reinterpret_cast<const T*>(a.kc), reinterpret_cast<const T*>(a.vc), head_base,
                          c * kAttnChunk, pos_last);
        __syncthreads();
#pragma unroll
        for (int rr = 0; rr < RPW; ++rr) {
            const int r = warp + kWarps * rr;
            if (r >= rows) break;
            const int t = t0 + r / n_rep;
            if (t >= a.tokens) continue;
            const int pos = base + t;
            if (c * kAttnChunk > pos) continue;
            const int jmax = min(kAttnChunk - 1, pos - c * kAttnChunk);
            float m, l, o[DPL];
            chunk_partial<T, DH>(qs + r * DH, Ks, Vs, jmax, a.scale_log2, m, l, o);
            if (c == 0) {
                M[rr] = m;
                L[rr] = l;
#pragma unroll
                for (int e = 0; e < DPL; ++e) O[rr][e] = o[e];
            } else {
                fold<DPL>(M[rr], L[rr], O[rr], m, l, o);
            }
        }
    }
    T* out = reinterpret_cast<T*>(a.o);
#pragma unroll
    for (int rr = 0; rr < RPW; ++rr) {
        const int r = warp + kWarps * rr;
        if (r >= rows) break;
        const int t = t0 + r / n_rep;
        if (t >= a.tokens) continue;
        const int h = g * n_rep + r % n_rep;
        T* dst = out + ((size_t)b * a.tokens + t) * qld + (size_t)h * DH + lane * DPL;
        const float inv_l = __frcp_rn(L[rr]);
#pragma unroll
        for (int e = 0; e < DPL; ++e) from_f(dst + e, __fmul_rn(O[rr][e], inv_l));
    }
}

// ----------------------------------------------------------------------------- decode
template <typename T, int DH>
__global__ void __launch_bounds__(kThreads) k_attn_decode_chunks(const AttnK a) {
    using TL = Tile<T, DH>;
    constexpr int DPL = TL::DPL;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    T* Ks = reinterpret_cast<T*>(smem_raw);
    T* Vs = Ks + kAttnChunk * TL::LD;
    float* qs = reinterpret_cast<float*>(Vs + kAttnChunk * TL::LD);

    ptx_wait();
    if (threadIdx.x == 0) ptx_launch_dependents();
    const int c = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    const int n_rep = a.n_heads / a.n_kv_heads;
    const int pos = base_position(a);
    if (pos < 0 || pos >= a.max_pos) {
        if (threadIdx.x == 0 && c == 0 && g == 0 && b == 0) record_error(a.err, LLAMA_ERR_POS_RANGE);
        return;
    }
    if (c * kAttnChunk > pos) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T* q = reinterpret_cast<const T*>(a.q);
    const size_t qld = (size_t)a.n_heads * DH;
    for (int i = threadIdx.x; i < n_rep * DH; i += kThreads) {
        const int r = i / DH, d = i % DH;
        qs[i] = to_f(q[(size_t)b * qld + (size_t)(g * n_rep + r) * DH + d]);
    }
    const size_t head_base = ((size_t)b * a.n_kv_heads + g) * a.kv_seq * DH;
    load_chunk<T, DH>(Ks, Vs, reinterpret_cast<const T*>(a.kc), reinterpret_cast<const T*>(a.vc), head_base,
                      c * kAttnChunk, pos);
    __syncthreads();
    const int jmax = min(kAttnChunk - 1, pos - c * kAttnChunk);
    for (int r = warp; r < n_rep; r += kWarps) {
        float m, l, o[DPL];
        chunk_partial<T, DH>(qs + r * DH, Ks, Vs, jmax, a.scale_log2, m, l, o);
        float* dst = a.partial + ((((size_t)b * a.n_kv_heads + g) * a.n_chunks + c) * n_rep + r) * part_stride(DH);
#pragma unroll
        for (int e = 0; e < DPL; ++e) dst[lane * DPL + e] = o[e];
        if (lane == 0) {
            dst[DH] = m;
            dst[DH + 1] = l;
        }
    }
}

template <typename T, int DH>
__global__ void __launch_bounds__(32) k_attn_decode_combine(const AttnK a) {
    TRACE(const unsigned long long tr0 = trace_stamp();)
    const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x;
    // The position is set before the step, never by the kernels this one overlaps.
    const int pos = a.pos_seq ? a.pos_seq[b] : base_position(a);
    // The O projection after this kernel reads only its weights before its own wait:
    // it may launch at once and take the SMs as the attention CTAs leave them.
    if (threadIdx.x == 0) ptx_launch_dependents();
    ptx_wait();
    TRACE(const unsigned long long tr1 = trace_stamp();)
    const int n_rep = a.n_heads / a.n_kv_heads;
    const int g = h / n_rep, r = h % n_rep;
    if (pos < 0 || pos >= a.max_pos) return;
    const float* base = a.partial + (((size_t)b * a.n_kv_heads + g) * a.n_chunks * n_rep + r) * part_stride(DH);
    T* dst = reinterpret_cast<T*>(a.o) + (size_t)b * a.n_heads * DH + (size_t)h * DH;
    fold_row<T, DH>(base, (size_t)n_rep * part_stride(DH), pos / kAttnChunk + 1, lane, dst);
    TRACE(trace_cta(TR_ATTN_COMBINE, tr0, tr1);)
}

// ----------------------------------------------------------------------------- decode on a paged cache
// The same chunk partial over keys whose rows are found through the block table: a
// chunk of 128 keys lies in 128 / page_size pages (one, from 128-key pages on).  Pages
// behind a sequence's last key are not looked up.  For the shapes the tensor-core kernel
// does not take: fp32, and groups of query heads that do not divide 128.
//
// Persistent: a CTA walks a contiguous range of the units (sequence, KV head, chunk),
// counted on the device from the lengths, so that a bound far above them costs nothing.
// K and V have a buffer each: the next unit's K is copied while this one's weights average
// V, its V while the next scores are taken.
struct PagedK {
    AttnK a;
    PageTable t;
    int pos_off;   // see paged_keys
    float2* part_ml;   // (m, l) of the partials (attn_paged_ml); a.partial: [b][head][chunk][DH]
};
constexpr int kPagedSeqs = 1024;   // sequences per launch of the chunk kernel

// WPR: warps per query row.  Small groups leave warps without a row, so a row's keys (of the
// scores) and columns (of the average) are then shared by two or four warps -- each score,
// weight and column is the same chain of operations, and a lane's four weights are added in
// the same order, so the bits stay those of chunk_partial.
template <typename T, int DH, int WPR>
__global__ void __launch_bounds__(kThreads, 2) k_attn_paged_chunks(const PagedK p) {
    using TL = Tile<T, DH>;
    constexpr int DPL = TL::DPL;
    constexpr int VPR = DH / TL::VEC;
    constexpr int RPW = WPR == 1 ? kRowsMax / kWarps : 1;   // rows per warp (WPR > 1: at most kWarps / WPR rows)
    constexpr int kCols = (DPL + WPR - 1) / WPR;            // columns lane + 32 k per lane, k = sub, sub + WPR, ...
    __shared__ __align__(16) float s_p[WPR == 1 ? 1 : kWarps / WPR][kAttnChunk];
    __shared__ float s_mx[kWarps];
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ int s_pre[kPagedSeqs + 1], s_keys[kPagedSeqs];   // units before each sequence, per KV head; its keys
    __shared__ int s_page[2][kAttnChunk / 16];
    T* Ks = reinterpret_cast<T*>(smem_raw);
    T* Vs = Ks + kAttnChunk * TL::LD;
    float* qs = reinterpret_cast<float*>(Vs + kAttnChunk * TL::LD);
    const AttnK& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_rep = a.n_heads / a.n_kv_heads;
    const int shift = p.t.shift, ps = 1 << shift;
    const int row = warp / WPR, sub = warp % WPR;   // WPR > 1

    ptx_wait();
    if (warp == 0) {
        int run = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 32) {
            const int b = b0 + lane;
            bool bad = false;
            const int keys = b < a.batch ? paged_keys(__ldcg(a.pos_seq + b), p.pos_off, a.max_pos, bad) : 0;
            int nt = (keys + kAttnChunk - 1) / kAttnChunk;
            if (b < a.batch) s_keys[b] = keys;
            if (bad && blockIdx.x == 0) record_error(a.err, LLAMA_ERR_POS_RANGE);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, nt, o);
                if (lane >= o) nt += v;
            }
            if (b < a.batch) s_pre[b + 1] = run + nt;
            run += __shfl_sync(kFull, nt, 31);
        }
        if (lane == 0) s_pre[0] = 0;
    }
    __syncthreads();
    const int n_units = s_pre[a.batch] * a.n_kv_heads;   // below 2^31: checked on the host from the bound
    const int u_begin = (int)((long)n_units * blockIdx.x / gridDim.x), u_end = (int)((long)n_units * (blockIdx.x + 1) / gridDim.x);

    struct Unit {
        int b, g, c, keys;   // keys of the sequence
    };
    auto unit = [&](int u) {
        Unit d;
        int lo = 0, hi = a.batch - 1;   // the last sequence whose units start at or before u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_pre[mid] * a.n_kv_heads <= u) lo = mid;
            else hi = mid - 1;
        }
        const int nt = s_pre[lo + 1] - s_pre[lo], r = u - s_pre[lo] * a.n_kv_heads;
        d.b = lo;
        d.g = r / nt;
        d.c = r - d.g * nt;
        d.keys = s_keys[lo];
        return d;
    };
    // the page ids of a unit's chunk (one thread each), visible after the next barrier
    auto lookup = [&](const Unit& d, int* pages) {
        const int key0 = d.c * kAttnChunk, n = (min(kAttnChunk, d.keys - key0) + ps - 1) >> shift;
        if (threadIdx.x < n) pages[threadIdx.x] = page_of(p.t, d.b, (key0 >> shift) + threadIdx.x, a.err);
    };
    auto copy = [&](const Unit& d, const int* pages, const void* cache, T* to) {
        const int key0 = d.c * kAttnChunk;
        for (int v = threadIdx.x; v < kAttnChunk * VPR; v += kThreads) {
            const int j = v / VPR, col = (v % VPR) * TL::VEC;
            const int key = key0 + j;
            const int page = key < d.keys ? pages[(key >> shift) - (key0 >> shift)] : -1;
            const size_t row = page < 0 ? 0 : (((size_t)page * a.n_kv_heads + d.g) << shift) + (key & (ps - 1));
            cp_async16(to + j * TL::LD + col, reinterpret_cast<const T*>(cache) + row * DH + col, page >= 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    if (u_begin >= u_end) return;
    Unit d = unit(u_begin);
    int turn = 0;   // of s_page
    lookup(d, s_page[0]);
    __syncthreads();
    copy(d, s_page[0], a.kc, Ks);
    copy(d, s_page[0], a.vc, Vs);
    int q_of = -1;   // (sequence, KV head) whose query rows are in qs
    for (int u = u_begin; u < u_end; ++u) {
        const bool more = u + 1 < u_end;
        Unit next = d;
        if (more) {
            next = unit(u + 1);
            lookup(next, s_page[turn ^ 1]);
        }
        if (d.b * a.n_kv_heads + d.g != q_of) {
            q_of = d.b * a.n_kv_heads + d.g;
            const T* q = reinterpret_cast<const T*>(a.q) + ((size_t)d.b * a.n_heads + (size_t)d.g * n_rep) * DH;
            for (int i = threadIdx.x; i < n_rep * DH; i += kThreads) qs[i] = to_f(q[i]);
        }
        asm volatile("cp.async.wait_group 1;" ::: "memory");   // K landed (this thread's part), V may not have
        __syncthreads();
        const int jmax = min(kAttnChunk - 1, d.keys - 1 - d.c * kAttnChunk);
        float w[RPW][4], m[RPW], l[RPW];
        if constexpr (WPR == 1) {
#pragma unroll
            for (int i = 0; i < RPW; ++i) {
                const int r = warp + i * kWarps;
                if (r < n_rep) chunk_weights<T, DH>(qs + r * DH, Ks, jmax, a.scale_log2, m[i], l[i], w[i]);
            }
        } else if (row < n_rep) {
            float s[4 / WPR], mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4 / WPR; ++i) {
                const int j = lane + 32 * (sub * (4 / WPR) + i);
                s[i] = j <= jmax ? __fmul_rn(key_dot<T, DH>(qs + row * DH, Ks + j * TL::LD), a.scale_log2) : -INFINITY;
                mx = fmaxf(mx, s[i]);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
            if (lane == 0) s_mx[warp] = mx;
            ptx::named_bar_sync(1 + row, 32 * WPR);
#pragma unroll
            for (int i = 0; i < WPR; ++i) mx = fmaxf(mx, s_mx[row * WPR + i]);
#pragma unroll
            for (int i = 0; i < 4 / WPR; ++i) {
                const int j = lane + 32 * (sub * (4 / WPR) + i);
                s_p[row][j] = j <= jmax ? exp2f(__fsub_rn(s[i], mx)) : 0.f;
            }
            ptx::named_bar_sync(1 + row, 32 * WPR);
            m[0] = mx;
            l[0] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) l[0] = __fadd_rn(l[0], s_p[row][lane + 32 * i]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) l[0] = __fadd_rn(l[0], __shfl_xor_sync(kFull, l[0], off));
        }
        __syncthreads();   // K was read
        if (more) copy(next, s_page[turn ^ 1], a.kc, Ks);
        else asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");   // V landed
        __syncthreads();
        if constexpr (WPR == 1) {
#pragma unroll
            for (int i = 0; i < RPW; ++i) {
                const int r = warp + i * kWarps;
                if (r >= n_rep) break;
                float o[DPL];
                chunk_average<T, DH>(Vs, jmax, w[i], o);
                const size_t slot = ((size_t)d.b * a.n_heads + (size_t)d.g * n_rep + r) * a.n_chunks + d.c;
#pragma unroll
                for (int e = 0; e < DPL; ++e) a.partial[slot * DH + lane * DPL + e] = o[e];
                if (lane == 0) p.part_ml[slot] = make_float2(m[i], l[i]);
            }
        } else if (row < n_rep && sub < DPL) {
            float o[kCols];
#pragma unroll
            for (int e = 0; e < kCols; ++e) o[e] = 0.f;
            const T* v = Vs + lane + 32 * sub;
            const float* wt = s_p[row];
            int j = 0;
            for (; j + 7 <= jmax; j += 8) {   // eight rows' words are read before the chain takes them
                float x[8][kCols], k[8];
#pragma unroll
                for (int t = 0; t < 8; t += 4) *reinterpret_cast<float4*>(k + t) = *reinterpret_cast<const float4*>(wt + j + t);
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int e = 0; e < kCols; ++e)
                        if (sub + e * WPR < DPL) x[t][e] = to_f(v[(j + t) * TL::LD + 32 * WPR * e]);
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int e = 0; e < kCols; ++e)
                        if (sub + e * WPR < DPL) o[e] = __fmaf_rn(k[t], x[t][e], o[e]);
            }
            for (; j <= jmax; ++j)
#pragma unroll
                for (int e = 0; e < kCols; ++e)
                    if (sub + e * WPR < DPL) o[e] = __fmaf_rn(wt[j], to_f(v[j * TL::LD + 32 * WPR * e]), o[e]);
            const size_t slot = ((size_t)d.b * a.n_heads + (size_t)d.g * n_rep + row) * a.n_chunks + d.c;
#pragma unroll
            for (int e = 0; e < kCols; ++e)
                if (sub + e * WPR < DPL) a.partial[slot * DH + lane + 32 * (sub + WPR * e)] = o[e];
            if (lane == 0 && sub == 0) p.part_ml[slot] = make_float2(m[0], l[0]);
        }
        __syncthreads();   // V was read
        if (more) copy(next, s_page[turn ^ 1], a.vc, Vs);
        d = next;
        turn ^= 1;
    }
}

// The combine of a paged call: a CTA per query row, whose chunks are folded in ascending
// order with the formula of attn_fold.cuh, bit for bit -- for any length.  A row's partials
// are contiguous ([chunk][DH], and [chunk] (m, l) apart), so a stage of 32 chunks arrives by
// one bulk copy, a ring of stages ahead, from a warp of its own.  The fold is a chain of one
// multiply-add per chunk and column once each chunk's two scales are known, and those need
// only the running maxima: the folding warps take them first, for up to kCombBlock chunks,
// from a prefix maximum.  A lane folds two columns: a warp alone on its scheduler is bound
// by its instructions and shared-memory reads per chunk (16 cycles; with one column a lane
// and four warps 24, with packed two-column arithmetic 26).
constexpr int kCombStage = 32;       // chunks per stage
constexpr int kCombStages = 8;       // at most
constexpr int kCombBlock = 1024;     // chunks whose scales are held at a time
constexpr int comb_threads(int dh) { return dh >= 64 ? dh / 2 : 32; }   // that fold

template <typename T, int DH>
__global__ void __launch_bounds__(comb_threads(DH) + 32) k_attn_paged_combine(const PagedK p, int n_stages, int n_scales) {
    constexpr int kThr = DH >= 64 ? DH / 2 : 32, kCol = DH / kThr, kPer = kCombBlock / kThr;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ float s_max[kThr / 32];
    __shared__ uint64_t s_full[kCombStages], s_empty[kCombStages];
    const AttnK& a = p.a;
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float* ring = reinterpret_cast<float*>(smem_raw);   // [stage][chunk][DH]
    // per chunk: scale of the past, of the chunk, l times the latter -- an array each, read four
    // chunks at a time
    float* scale = ring + (size_t)n_stages * kCombStage * DH;
    // what wrote the lengths has completed: the kernel before this one starts it only after its
    // own wait
    bool bad;
    const int keys = paged_keys(a.pos_seq[b], p.pos_off, a.max_pos, bad);
    if (tid == 0) {
        for (int i = 0; i < n_stages; ++i) {
            ptx::mbar_init(&s_full[i], 1);
            ptx::mbar_init(&s_empty[i], kThr / 32);
        }
        ptx::fence_mbar_init();
        ptx_launch_dependents();
    }
    __syncthreads();
    ptx_wait();
    T* dst = reinterpret_cast<T*>(a.o) + ((size_t)b * a.n_heads + h) * DH + tid * kCol;
    if (keys == 0) {   // no key to attend: a row of zeros
        if (warp < kThr / 32)
#pragma unroll
            for (int e = 0; e < kCol; ++e) from_f(dst + e, 0.f);
        return;
    }
    const int n_chunks = (keys - 1) / kAttnChunk + 1;
    const size_t row = ((size_t)b * a.n_heads + h) * a.n_chunks;   // (KV head, query row of its group) is the head
    if (warp == kThr / 32) {
        if (lane == 0) {
            const float* part = a.partial + row * DH;
            const int stages = (n_chunks + kCombStage - 1) / kCombStage;
            int issued = 0;
            for (; issued < stages; ++issued) {
                const int at = issued % n_stages, n = min(kCombStage, n_chunks - issued * kCombStage);
                if (issued >= n_stages && !ptx::mbar_wait(&s_empty[at], (issued / n_stages - 1) & 1, a.err)) break;
                ptx::mbar_arrive_expect_tx(&s_full[at], n * DH * 4);
                ptx::bulk_load(ring + (size_t)at * kCombStage * DH, part + (size_t)issued * kCombStage * DH, n * DH * 4,
                               &s_full[at]);
            }
            // no copy may still be landing when the CTA leaves (all have landed unless a wait gave up)
            for (int i = max(0, issued - n_stages); i < issued; ++i)
                ptx::mbar_wait_drain(&s_full[i % n_stages], (i / n_stages) & 1);
        }
        return;
    }
    const float2* part_ml = p.part_ml + row;
    // -0 + x == x for every x: the first chunk's scales (0, 1) give its partial itself
    float M = -INFINITY, L = -0.f, O[2] = {-0.f, -0.f};
    bool ok = true;
    int at = 0, turn = 0;   // place in the ring, its parity
    for (int block = 0; block < n_chunks; block += kCombBlock) {
        const int nb = min(kCombBlock, n_chunks - block), per = (nb + kThr - 1) / kThr;
        // this thread's chunks: block + tid * per + i, i < per <= N
        auto take_scales = [&](auto count) {
            constexpr int N = decltype(count)::value;
            float m[N], l[N], most = -INFINITY;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = tid * per + i;
                const float2 ml = i < per && c < nb ? __ldcg(part_ml + block + c) : make_float2(-INFINITY, 0.f);
                m[i] = ml.x;
                l[i] = ml.y;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) most = fmaxf(most, m[i]);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float v = __shfl_up_sync(kFull, most, o);
                if (lane >= o) most = fmaxf(most, v);
            }
            ptx::named_bar_sync(1, kThr);   // the maxima and scales of the block before were read
            if (lane == 31) s_max[warp] = most;
            ptx::named_bar_sync(1, kThr);
            float now = __shfl_up_sync(kFull, most, 1);
            if (lane == 0) now = -INFINITY;
            now = fmaxf(M, now);
#pragma unroll
            for (int w = 0; w < kThr / 32; ++w) {
                if (w < warp) now = fmaxf(now, s_max[w]);
                M = fmaxf(M, s_max[w]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = tid * per + i;
                if (i < per && c < nb) {
                    const bool first = block + c == 0;
                    const float next = fmaxf(now, m[i]);
                    const float sa = first ? 0.f : exp2f(__fsub_rn(now, next)), sb = first ? 1.f : exp2f(__fsub_rn(m[i], next));
                    scale[c] = sa;
                    scale[n_scales + c] = sb;
                    scale[2 * n_scales + c] = __fmul_rn(l[i], sb);
                    now = next;
                }
            }
            ptx::named_bar_sync(1, kThr);
        };
        // short rows are not made to walk the longest one's unrolled rounds (1 us of a call)
        if (per == 1) take_scales(std::integral_constant<int, 1>{});
        else if (per <= 4) take_scales(std::integral_constant<int, 4>{});
        else take_scales(std::integral_constant<int, kPer>{});
        for (int c0 = 0; c0 < nb; c0 += kCombStage) {
            const int n = min(kCombStage, nb - c0);
            ok = ok && ptx::mbar_wait(&s_full[at], turn, a.err);
            const float* st = ring + (size_t)at * kCombStage * DH + tid * kCol;
            const float* k = scale + c0;
            auto step = [&](float ka, float kb, float kl, const float* x) {
                L = __fmaf_rn(L, ka, kl);
                if constexpr (kCol == 2) {
                    const float2 v = *reinterpret_cast<const float2*>(x);
                    O[0] = __fmaf_rn(O[0], ka, __fmul_rn(v.x, kb));
                    O[1] = __fmaf_rn(O[1], ka, __fmul_rn(v.y, kb));
                } else {
                    O[0] = __fmaf_rn(O[0], ka, __fmul_rn(x[0], kb));
                }
            };
            if (n == kCombStage) {
#pragma unroll
                for (int c = 0; c < kCombStage; c += 4) {
                    const float4 ka = *reinterpret_cast<const float4*>(k + c);
                    const float4 kb = *reinterpret_cast<const float4*>(k + n_scales + c);
                    const float4 kl = *reinterpret_cast<const float4*>(k + 2 * n_scales + c);
                    step(ka.x, kb.x, kl.x, st + c * DH);
                    step(ka.y, kb.y, kl.y, st + (c + 1) * DH);
                    step(ka.z, kb.z, kl.z, st + (c + 2) * DH);
                    step(ka.w, kb.w, kl.w, st + (c + 3) * DH);
                }
            } else {
#pragma unroll 4
                for (int c = 0; c < n; ++c) step(k[c], k[n_scales + c], k[2 * n_scales + c], st + c * DH);
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s_empty[at]);
            if (++at == n_stages) {
                at = 0;
                turn ^= 1;
            }
        }
    }
    if (!ok) return;   // a wait gave up (recorded)
    const float inv = __frcp_rn(L);
#pragma unroll
    for (int e = 0; e < kCol; ++e) from_f(dst + e, __fmul_rn(O[e], inv));
}

template <typename T, int DH>
size_t smem_bytes(int rows) {
    return 2 * (size_t)kAttnChunk * Tile<T, DH>::LD * sizeof(T) + (size_t)rows * DH * sizeof(float);
}

AttnK make_k(const AttnArgs& a) {
    AttnK k{};
    k.q = a.q;
    k.o = a.o;
    k.kc = a.kc;
    k.vc = a.vc;
    k.batch = a.batch;
    k.tokens = a.tokens;
    k.n_heads = a.n_heads;
    k.n_kv_heads = a.n_kv_heads;
    k.kv_seq = a.kv_seq;
    k.start_pos = a.start_pos;
    k.max_pos = a.max_pos;
    k.pos_dev = a.pos_dev;
    k.pos_seq = a.pos_seq;
    k.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)a.head_dim));
    k.partial = a.partial;
    k.n_chunks = a.n_chunks;
    k.err = a.err;
    return k;
}

template <typename T, int DH>
cudaError_t combine_launch(const AttnK& k, cudaStream_t s) {
    auto kern = k_attn_decode_combine<T, DH>;
    cudaError_t r = kernel_setup_once((const void*)kern, setup_prefer_shared);
    if (r != cudaSuccess) return r;
    return launch_pdl(kern, dim3(k.n_heads, k.batch), dim3(32), 0, s, k);
}

template <typename T, int DH>
cudaError_t prefill_impl(const AttnArgs& a, cudaStream_t s) {
    AttnK k = make_k(a);
    const int n_rep = a.n_heads / a.n_kv_heads;
    k.tq = kRowsMax / n_rep;
    if (k.tq < 1) return cudaErrorInvalidValue;
    const size_t sm = smem_bytes<T, DH>(kRowsMax);
    auto kern = k_attn_prefill<T, DH>;
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
    if (r != cudaSuccess) return r;
    dim3 grid((a.tokens + k.tq - 1) / k.tq, a.n_kv_heads, a.batch);
    return launch_pdl(kern, grid, dim3(kThreads), sm, s, k);
}

template <typename T, int DH>
cudaError_t decode_impl(const AttnArgs& a, cudaStream_t s) {
    AttnK k = make_k(a);
    const int n_rep = a.n_heads / a.n_kv_heads;
    const size_t sm = smem_bytes<T, DH>(n_rep);
    auto kern = k_attn_decode_chunks<T, DH>;
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
    if (r != cudaSuccess) return r;
    dim3 grid(a.n_chunks, a.n_kv_heads, a.batch);
    r = launch_pdl(kern, grid, dim3(kThreads), sm, s, k);
    if (r != cudaSuccess) return r;
    return combine_launch<T, DH>(k, s);
}

template <typename T, int DH>
cudaError_t combine_impl(const AttnArgs& a, cudaStream_t s) {
    return combine_launch<T, DH>(make_k(a), s);
}

PagedK make_paged(const AttnArgs& a) {
    PagedK p{};
    p.a = make_k(a);
    p.t = a.pages;
    p.pos_off = a.pos_off;
    p.part_ml = attn_paged_ml(a.partial, a.batch, a.n_heads, a.n_chunks, a.head_dim);
    return p;
}

template <typename T, int DH>
cudaError_t paged_combine_impl(const AttnArgs& a, cudaStream_t s) {
    auto kern = k_attn_paged_combine<T, DH>;
    constexpr int kStage = kCombStage * DH * (int)sizeof(float), kScale = 3 * (int)sizeof(float);
    cudaError_t r = kernel_setup_once((const void*)kern, [](const void* k) {
        cudaError_t e = setup_prefer_shared(k);
        return e != cudaSuccess ? e
                                : cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       kCombStages * kStage + kCombBlock * kScale);
    });
    if (r != cudaSuccess) return r;
    // A ring for the longest row there can be.  One or two stages hold most decode lengths,
    // and the more CTAs an SM takes the more rows are in flight; beyond that half a ring, or
    // all of it where every row has an SM to itself.
    const int need = (a.n_chunks + kCombStage - 1) / kCombStage;
    const int most = (long)a.n_heads * a.batch <= device_sm_count() ? kCombStages : kCombStages / 2;
    const int n_stages = std::min(need, most), scales = std::min(need * kCombStage, kCombBlock);
    return launch_pdl(kern, dim3(a.n_heads, a.batch), dim3(comb_threads(DH) + 32), n_stages * kStage + scales * kScale, s,
                      make_paged(a), n_stages, scales);
}

template <typename T, int DH, int WPR>
cudaError_t paged_chunks_launch(const AttnArgs& a, cudaStream_t s) {
    auto kern = k_attn_paged_chunks<T, DH, WPR>;
    cudaError_t r = kernel_setup_once((const void*)kern, [](const void* k) {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<T, DH>(kRowsMax));
    });
    if (r != cudaSuccess) return r;
    const int n_rep = a.n_heads / a.n_kv_heads;
    const size_t smem = smem_bytes<T, DH>(n_rep);
    const int per_sm = smem <= 100 * 1024 ? 2 : 1;   // two CTAs by their registers
    for (int b0 = 0; b0 < a.batch; b0 += kPagedSeqs) {
        PagedK k = make_paged(a);
        k.a.batch = std::min(a.batch - b0, kPagedSeqs);
        k.a.pos_seq += b0;
        k.t.table += (size_t)b0 * a.pages.stride;
        k.a.q = (const T*)a.q + (size_t)b0 * a.n_heads * DH;
        k.a.partial += (size_t)b0 * a.n_heads * a.n_chunks * DH;
        k.part_ml += (size_t)b0 * a.n_heads * a.n_chunks;
        const long max_units = (long)k.a.batch * a.n_kv_heads * a.n_chunks;
        const dim3 grid((unsigned)std::min<long>(max_units, (long)device_sm_count() * per_sm));
        r = launch_pdl(kern, grid, dim3(kThreads), smem, s, k);
        if (r != cudaSuccess) return r;
    }
    return cudaSuccess;
}

template <typename T, int DH>
cudaError_t paged_decode_impl(const AttnArgs& a, cudaStream_t s) {
    const int n_rep = a.n_heads / a.n_kv_heads;
    // warps per row: as many as leave every row of the group its own
    const cudaError_t r = n_rep <= kWarps / 4   ? paged_chunks_launch<T, DH, 4>(a, s)
                          : n_rep <= kWarps / 2 ? paged_chunks_launch<T, DH, 2>(a, s)
                                                : paged_chunks_launch<T, DH, 1>(a, s);
    return r != cudaSuccess ? r : paged_combine_impl<T, DH>(a, s);
}

}  // namespace

LLAMA_TRACE_UNIT(attn_simt)

cudaError_t launch_attention_paged_combine(const AttnArgs& a, cudaStream_t s) {
    if (a.dtype == LLAMA_BF16) return a.head_dim == 128 ? paged_combine_impl<bf16, 128>(a, s) : cudaErrorInvalidValue;
    switch (a.head_dim) {
        case 32: return paged_combine_impl<float, 32>(a, s);
        case 64: return paged_combine_impl<float, 64>(a, s);
        case 128: return paged_combine_impl<float, 128>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_attention_paged(const AttnArgs& a, cudaStream_t s) {
    if (a.batch <= 0) return cudaSuccess;
    // where the contiguous decode takes the tensor cores
    if (a.dtype == LLAMA_BF16 && attention_tc_supported(a.n_heads, a.n_kv_heads, a.head_dim))
        return launch_attention_tc_paged(a, s);
    if (a.dtype == LLAMA_BF16) return a.head_dim == 128 ? paged_decode_impl<bf16, 128>(a, s) : cudaErrorInvalidValue;
    switch (a.head_dim) {
        case 32: return paged_decode_impl<float, 32>(a, s);
        case 64: return paged_decode_impl<float, 64>(a, s);
        case 128: return paged_decode_impl<float, 128>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

size_t attn_decode_partial_bytes(int batch, int n_kv_heads, int n_chunks, int n_rep, int head_dim) {
    return (size_t)batch * n_kv_heads * n_chunks * n_rep * part_stride(head_dim) * sizeof(float);
}

cudaError_t launch_attention_combine(const AttnArgs& a, cudaStream_t s) {
    if (a.batch <= 0) return cudaSuccess;
    if (a.dtype == LLAMA_BF16) {
        if (a.head_dim == 128) return combine_impl<bf16, 128>(a, s);
        return cudaErrorInvalidValue;
    }
    switch (a.head_dim) {
        case 32: return combine_impl<float, 32>(a, s);
        case 64: return combine_impl<float, 64>(a, s);
        case 128: return combine_impl<float, 128>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_attention_prefill(const AttnArgs& a, cudaStream_t s) {
    if (a.batch <= 0 || a.tokens <= 0) return cudaSuccess;
    if (a.dtype == LLAMA_BF16) {
        if (a.head_dim == 128) return prefill_impl<bf16, 128>(a, s);
        return cudaErrorInvalidValue;
    }
    switch (a.head_dim) {
        case 32: return prefill_impl<float, 32>(a, s);
        case 64: return prefill_impl<float, 64>(a, s);
        case 128: return prefill_impl<float, 128>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_attention_decode(const AttnArgs& a, cudaStream_t s) {
    if (a.batch <= 0) return cudaSuccess;
    if (a.dtype == LLAMA_BF16) {
        if (a.head_dim == 128) return decode_impl<bf16, 128>(a, s);
        return cudaErrorInvalidValue;
    }
    switch (a.head_dim) {
        case 32: return decode_impl<float, 32>(a, s);
        case 64: return decode_impl<float, 64>(a, s);
        case 128: return decode_impl<float, 128>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace llama
