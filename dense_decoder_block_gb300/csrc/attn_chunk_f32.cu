// Attention of chunks of new tokens over a paged cache in fp32 on the CUDA cores (head_dim 32, 64, 128).
//
// A tile is up to 64 query rows of a KV group; its keys come in blocks of 64, two buffers, the next block's copies
// (cp.async, 16 bytes a thread) under the arithmetic of this one.  256 threads: thread (y, x) of 16 x 16 holds rows 4y ..
// 4y + 3 and keys x, x + 16, x + 32, x + 48 of a block's scores, and columns of O: 8 scalar products' multiply-adds for
// each 16-byte read of shared memory.  A row's maximum and sum run over its 16 threads by shuffles; O is scaled where the
// maximum moves, and every kF32Carry blocks O and l are added to second sums (attn_chunk.cuh).  Bound by the multiply-adds
// and the reads that feed them; tiles are split over the CTAs and joined as attn_chunk.cuh says, since a chunk of a tile
// takes microseconds.  2048 tokens of 8 / 2 heads of 128: 278 us (31 TFLOP/s); 8 x 64 behind 2000, 8 / 2 heads of 64: 100;
// 2 x 16 behind 4: 10 in a graph, round trips.
#include <algorithm>

#include "attn_chunk.cuh"
#include "internal.h"

namespace llama {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = kF32Rows, kKeys = kF32Keys;
constexpr int kGroupBlocks = 4;   // blocks of a piece from which on idle warps share its keys

template <int DH>
struct Tile {
    static constexpr int LD = DH + 4;                    // padded rows of Q, K (reads along a row, 16 rows apart in a warp)
    static constexpr int LDP = kKeys + 4;
    static constexpr int OFF_K = kRows * LD;             // floats; [buffer]
    static constexpr int OFF_V = OFF_K + 2 * kKeys * LD;
    static constexpr int OFF_P = OFF_V + 2 * kKeys * DH;
    static constexpr int OFF_IDS = OFF_P + kRows * LDP;  // [block % 4][4]: its pages, 16 rows each at least
    static constexpr int OFF_CARRY = OFF_IDS + 16;       // [row] (m, l) of what was carried over
    static constexpr int OFF_SEQS = OFF_CARRY + 2 * kRows;
    static constexpr int BYTES = OFF_SEQS * 4 + (int)sizeof(ChunkSeqs<kF32Seqs>);
    static constexpr int VPR = DH / 4;                   // vectors per row
    static constexpr int CPT = DH / 16;                  // columns of O per thread
    static constexpr int CTAS = f32_ctas_per_sm(DH);     // per SM
};

__device__ __forceinline__ void cp_async16(void* smem, const void* gmem, bool valid) {
    const int src = valid ? 16 : 0;   // 0: zeros, nothing read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(smem)), "l"(gmem), "r"(src) : "memory");
}

// Sum and maximum over the 16 threads of a row.
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int DH>
__global__ void __launch_bounds__(kThreads, Tile<DH>::CTAS) k_attn_chunk_f32(const ChunkArgs a) {
    using TL = Tile<DH>;
    constexpr int CPT = TL::CPT;
    extern __shared__ __align__(16) float sm[];
    using Seqs = ChunkSeqs<kF32Seqs>;
    Seqs& seqs = *reinterpret_cast<Seqs*>(sm + TL::OFF_SEQS);
    const int tid = threadIdx.x, x = tid & 15;
    ptx::griddep_wait();
    if (tid < 32) chunk_seqs(a, seqs, blockIdx.x == 0);
    __syncthreads();
    const int n_rep = a.n_heads / a.n_kv_heads, shift = a.pages.shift;
    ChunkWalk walk(a, seqs, blockIdx.x, gridDim.x);
    if (tid < 32) walk.begin(a);
    if (tid == 0) ptx::griddep_launch_dependents();
    ChunkPiece p;
    while (walk.next(p)) {
        const int rows = (p.t1 - p.t0) * n_rep;
        const int key_end = min(p.c1 * kAttnChunk, p.kv_last + 1), blocks = (key_end - p.c0 * kAttnChunk + kKeys - 1) / kKeys;
        // the pages of block i, looked up two blocks ahead of their copies (a look-up in front of each copy: the call
        // 45 us, so 41.6; 1 token behind 4000, 8 heads of 128)
        int* ids = reinterpret_cast<int*>(sm + TL::OFF_IDS);
        auto look_up = [&](int i, int k) {
            const int key = p.c0 * kAttnChunk + i * kKeys + (k << min(shift, 6));
            if (k < max(kKeys >> shift, 1) && key < key_end) ids[(i & 3) * 4 + k] = max(page_of(a.pages, p.b, key >> shift, a.err), 0);
        };
        // keys of block i into buffer i % 2; a thread's vectors: column tid % VPR of rows tid / VPR, ...
        auto copy = [&](int i) {
            if (tid < 4) look_up(i + 2, tid);
            const int key0 = p.c0 * kAttnChunk + i * kKeys;
            float* ks = sm + TL::OFF_K + (i & 1) * kKeys * TL::LD;
            float* vs = sm + TL::OFF_V + (i & 1) * kKeys * DH;
            for (int e = tid; e < kKeys * TL::VPR; e += kThreads) {
                const int r = e / TL::VPR, c = e % TL::VPR * 4, key = key0 + r;
                const bool in = key < key_end;
                size_t at = 0;
                if (in) {
                    const int id = ids[(i & 3) * 4 + (r >> shift)];   // blocks of 64 lie in one page of 64 or more
                    at = ((((size_t)id * a.n_kv_heads + p.g) << shift) + (key & ((1 << shift) - 1))) * DH + c;
                }
                cp_async16(ks + r * TL::LD + c, static_cast<const float*>(a.kc) + at, in);
                cp_async16(vs + r * DH + c, static_cast<const float*>(a.vc) + at, in);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        __syncthreads();   // the last piece's buffers are used up
        if (tid < 8) look_up(tid >> 2, tid & 3);
        __syncthreads();
        copy(0);
        for (int e = tid; e < kRows * TL::VPR; e += kThreads) {
            const int r = e / TL::VPR, c = e % TL::VPR * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int t = p.t0 + r / n_rep, h = p.g * n_rep + r % n_rep;
                v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                                     (((size_t)p.b * a.tokens + t) * a.n_heads + h) * DH + c);
            }
            *reinterpret_cast<float4*>(sm + r * TL::LD + c) = v;
        }
        // 8 rows a warp; the warps that few rows leave over take a block's keys between them: group g of G the keys
        // 64 g / G .. of every block, each group with a softmax of its own, joined at the end (1 token behind 4000, 8 heads of
        // 128: 41.6 -> 32.4 us; joining costs 2 us, so not for few blocks)
        const int groups = blocks < kGroupBlocks ? 1 : rows <= 16 ? 4 : rows <= 32 ? 2 : 1, warps = 8 / groups;
        const int group = (tid >> 5) / warps, y = 2 * ((tid >> 5) % warps) + (tid >> 4 & 1);
        const bool live = 8 * (y >> 1) < rows;
        // this thread's rows 4y .. 4y + 3: last key that each sees (-1: no row)
        int last[4];
        float m[4], l[4], o[4][CPT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * y + i;
            last[i] = r < rows ? p.pos0 + r / n_rep : -1;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < CPT; ++e) o[i][e] = 0.f;
        }
        // O and l to the sums in the workspace and in shared memory (relative to each row's maximum then), the same threads'
        // every time; they begin anew.  Rows of group g at kRows / groups * g.
        const int carry_row = kRows / groups * group + 4 * y;
        float* carry = a.carry + (size_t)blockIdx.x * (kRows * DH) + carry_row * DH + x * CPT;
        float2* carried = reinterpret_cast<float2*>(sm + TL::OFF_CARRY) + carry_row;
        auto carry_over = [&](bool first) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 before = carried[i];
                const float w = before.x == -INFINITY ? 0.f : exp2f(before.x - m[i]);
                if (!first) l[i] = __fmaf_rn(before.y, w, l[i]);
#pragma unroll
                for (int e = 0; e < CPT; e += 2) {
                    float2* to = reinterpret_cast<float2*>(carry + i * DH + e);
                    float2 sum = make_float2(o[i][e], o[i][e + 1]);
                    if (!first) {
                        const float2 z = __ldcg(to);
                        sum = make_float2(__fmaf_rn(z.x, w, sum.x), __fmaf_rn(z.y, w, sum.y));
                    }
                    __stcg(to, sum);
                    o[i][e] = o[i][e + 1] = 0.f;
                }
                __syncwarp();
                if (x == 0) carried[i] = make_float2(m[i], l[i]);
                l[i] = 0.f;
            }
            __syncwarp();
        };
        for (int i0 = 0; i0 < blocks; ++i0) {
            if (i0 + 1 < blocks) {
                copy(i0 + 1);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncthreads();
            if (i0 > 0 && i0 % kF32Carry == 0 && live) carry_over(i0 == kF32Carry);
            const float* ks = sm + TL::OFF_K + (i0 & 1) * kKeys * TL::LD;
            const float* vs = sm + TL::OFF_V + (i0 & 1) * kKeys * DH;
            const int key0 = p.c0 * kAttnChunk + i0 * kKeys;
            if (!live) {   // no row in this warp (few new tokens)
                __syncthreads();
                continue;
            }
            auto block = [&](auto of) {   // JN times 16 keys
                constexpr int JN = decltype(of)::value;
                const int j0 = group * JN;
                float s[4][JN] = {};
#pragma unroll 4
                for (int d = 0; d < DH; d += 4) {
                    float4 q[4], k[JN];
#pragma unroll
                    for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const float4*>(sm + (4 * y + i) * TL::LD + d);
#pragma unroll
                    for (int j = 0; j < JN; ++j) k[j] = *reinterpret_cast<const float4*>(ks + (x + 16 * (j0 + j)) * TL::LD + d);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < JN; ++j)
                            s[i][j] = __fmaf_rn(q[i].w, k[j].w, __fmaf_rn(q[i].z, k[j].z, __fmaf_rn(q[i].y, k[j].y, __fmaf_rn(q[i].x, k[j].x, s[i][j]))));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int j = 0; j < JN; ++j) {
                        s[i][j] = key0 + x + 16 * (j0 + j) <= last[i] ? s[i][j] * a.scale_log2 : -INFINITY;
                        mx = fmaxf(mx, s[i][j]);
                    }
                    const float mn = fmaxf(m[i], row_max(mx)), ref = mn == -INFINITY ? 0.f : mn;
                    const float c = exp2f(m[i] - ref);   // m = -inf: 0
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < JN; ++j) {
                        const float w = key0 + x + 16 * (j0 + j) <= last[i] ? exp2f(s[i][j] - ref) : 0.f;
                        sm[TL::OFF_P + (4 * y + i) * TL::LDP + x + 16 * (j0 + j)] = w;
                        sum += w;
                    }
                    l[i] = __fmaf_rn(l[i], c, row_sum(sum));
                    m[i] = mn;
#pragma unroll
                    for (int e = 0; e < CPT; ++e) o[i][e] *= c;
                }
                __syncwarp();   // a warp's rows of P are its own
                // a row does not see what lies behind it, infinities and NaN included: such products are left out
                const bool all = key0 + kKeys - 1 <= p.pos0;
                auto average = [&](auto masked) {
                    constexpr bool kMasked = decltype(masked)::value;
                    // (20 keys: the call 12.8 -> 11.4 us)
                    const int k1 = kMasked ? min(16 * (j0 + JN), key_end - key0) : 16 * (j0 + JN);
#pragma unroll 2
                    for (int k = 16 * j0; k < k1; k += 4) {
                        float4 w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(sm + TL::OFF_P + (4 * y + i) * TL::LDP + k);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            float v[CPT];
                            if constexpr (CPT >= 4) {
#pragma unroll
                                for (int e = 0; e < CPT; e += 4)   // columns 4x .. 4x + 3 of each 64
                                    *reinterpret_cast<float4*>(v + e) = *reinterpret_cast<const float4*>(vs + (k + kk) * DH + e * 16 + 4 * x);
                            } else {
                                *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(vs + (k + kk) * DH + 2 * x);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float wi = kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
                                const bool sees = !kMasked || key0 + k + kk <= last[i];
#pragma unroll
                                for (int e = 0; e < CPT; ++e)
                                    if (sees) o[i][e] = __fmaf_rn(wi, v[e], o[i][e]);
                            }
                        }
                    }
                };
                if (all) average(std::false_type{});
                else average(std::true_type{});
            };
            if (groups == 1) block(std::integral_constant<int, 4>{});
            else if (groups == 2) block(std::integral_constant<int, 2>{});
            else block(std::integral_constant<int, 1>{});
            __syncthreads();   // the buffer may be filled again
        }
        if (blocks > kF32Carry && live) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 before = carried[i];
                const float w = before.x == -INFINITY ? 0.f : exp2f(before.x - m[i]);
                l[i] = __fmaf_rn(before.y, w, l[i]);
#pragma unroll
                for (int e = 0; e < CPT; ++e) o[i][e] = __fmaf_rn(__ldcg(carry + i * DH + e), w, o[i][e]);
            }
        }
        if (groups > 1) {
            // [group][row] m, l and o, over K's buffers (as many values as one holds): group 0 joins
            float* os = sm + TL::OFF_K;
            float2* mls = reinterpret_cast<float2*>(sm + TL::OFF_P);
            const int per = kRows / groups;
            auto column = [&](int e) { return CPT >= 4 ? (e >> 2) * 64 + 4 * x + (e & 3) : 2 * x + e; };
            if (live && group > 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (x == 0) mls[group * per + 4 * y + i] = make_float2(m[i], l[i]);
#pragma unroll
                    for (int e = 0; e < CPT; ++e) os[(group * per + 4 * y + i) * DH + column(e)] = o[i][e];
                }
            }
            __syncthreads();
            if (group > 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * y + i >= rows) break;
                float M = m[i];
                for (int g = 1; g < groups; ++g) M = fmaxf(M, mls[g * per + 4 * y + i].x);
                // m = -inf: 0 (a NaN in l or o stays)
                float c = m[i] == -INFINITY ? 0.f : exp2f(m[i] - M);
                l[i] *= c;
#pragma unroll
                for (int e = 0; e < CPT; ++e) o[i][e] *= c;
                for (int g = 1; g < groups; ++g) {
                    const float2 ml = mls[g * per + 4 * y + i];
                    c = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
                    l[i] = __fmaf_rn(ml.y, c, l[i]);
#pragma unroll
                    for (int e = 0; e < CPT; ++e) o[i][e] = __fmaf_rn(os[(g * per + 4 * y + i) * DH + column(e)], c, o[i][e]);
                }
                m[i] = M;
            }
        }
        const bool split = p.c1 - p.c0 < p.n;
        const int slot = 2 * blockIdx.x + (p.c0 == 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * y + i;
            if (r >= rows) continue;
            const int t = p.t0 + r / n_rep, h = p.g * n_rep + r % n_rep;
            const float inv = split ? 1.f : 1.f / l[i];
            float* dst = static_cast<float*>(a.o) + (((size_t)p.b * a.tokens + t) * a.n_heads + h) * DH;
            float* part = a.partial + (size_t)slot * (kRows * DH);   // [column / 4][row][4]
            if (split && x == 0) a.part_ml[slot * kRows + r] = make_float2(m[i], l[i]);
            constexpr int W = CPT >= 4 ? 4 : 2;
#pragma unroll
            for (int e = 0; e < CPT; e += W) {
                const int col = e * 16 + W * x;
                float* to = split ? part + (col >> 2) * (kRows * 4) + r * 4 + (col & 3) : dst + col;
                if constexpr (W == 4)
                    *reinterpret_cast<float4*>(to) = make_float4(o[i][e] * inv, o[i][e + 1] * inv, o[i][e + 2] * inv, o[i][e + 3] * inv);
                else
                    *reinterpret_cast<float2*>(to) = make_float2(o[i][e] * inv, o[i][e + 1] * inv);
            }
        }
    }
}

template <int DH>
cudaError_t launch(const ChunkArgs& a, cudaStream_t s) {
    using TL = Tile<DH>;
    const auto kern = k_attn_chunk_f32<DH>;
    cudaError_t r = kernel_setup_once((const void*)kern, [](const void* k) {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Tile<DH>::BYTES);
    });
    if (r != cudaSuccess) return r;
    for (int b0 = 0; b0 < a.batch; b0 += kF32Seqs) {
        ChunkArgs k = a;
        const size_t at = (size_t)b0 * a.tokens * a.n_heads * DH;
        k.batch = std::min(a.batch - b0, kF32Seqs);
        k.q = static_cast<const float*>(a.q) + at;
        k.o = static_cast<float*>(a.o) + at;
        k.start += b0;
        k.count += b0;
        k.pages.table += (size_t)b0 * a.pages.stride;
        const unsigned n_ctas = (unsigned)std::min(device_sm_count() * TL::CTAS, kF32Ctas / 2 * TL::CTAS);
        r = launch_pdl(kern, dim3(n_ctas), dim3(kThreads), Tile<DH>::BYTES, s, k);
        if (r != cudaSuccess) return r;
        if (n_ctas == 1 || a.max_pos < kNeverSplit) continue;
        r = launch_pdl(k_attn_chunk_join<float, DH, 1, kRows>, dim3(4 * n_ctas), dim3(kJoinThreads), 0, s, k, (int)n_ctas);
        if (r != cudaSuccess) return r;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_chunk_f32(const ChunkArgs& a, int head_dim, cudaStream_t s) {
    switch (head_dim) {
        case 32: return launch<32>(a, s);
        case 64: return launch<64>(a, s);
        case 128: return launch<128>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace llama
