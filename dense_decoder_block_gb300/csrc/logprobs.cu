// llama_token_logprobs: log probabilities of given tokens, entropy and top alternatives of fp32 logits.
//
// With m = max z = z_u (u the first such token) and e_v = e^(z_v - m), d = sum_{v != u} e_v and
// t = sum e_v (z_v - m) (terms of weight 0 left out):
//   log p_v = (z_v - m) - log(1 + d),   H = log(1 + d) - t / (1 + d),
// all without cancellation: the terms of t are <= 0, and leaving the 1 out of the sums keeps small d.
//
// One pass over the logits.  A row is cut into segments of kSeg logits; a warp takes a segment at a time, all its
// loads issued ahead, and keeps per lane the running maximum, d and t relative to it (the maximum's own term left out),
// and per segment the maximum.  The lanes' triples are joined in fp64.  The n largest logits lie in the n segments with
// the largest maxima (equal maxima: the first segments): a segment outside has n segments whose best is better than all
// it has.  So the alternatives come from n segments read a second time, from L2.
//
// Few rows are split over a cluster of CTAs (their triples and segment maxima in distributed shared memory, the first
// CTA finishes the row), many rows take a CTA each.
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int kMaxTop = 32;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kVec = 4;                        // 16-byte vectors of a lane in a segment
constexpr int kSeg = 32 * 4 * kVec;            // 512 logits
constexpr int kMaxSegs = (1 << 20) / kSeg + 1; // of a row (one more where it starts off 16 bytes)
constexpr int kMaxCluster = 8;

struct LogprobArgs {
    const float* logits;
    int rows, vocab, n_top;
    const int* tokens;
    float* logprobs;
    float* entropy;
    int* top_ids;
    float* top_logprobs;
    int* err;
};

// Order of logits: larger first, equal ones by increasing place; a NaN counts as the lowest value, so that every order
// is total.
__device__ __forceinline__ unsigned order_bits(float z) {
    if (!(z == z)) z = -INFINITY;
    const unsigned u = __float_as_uint(z + 0.f);   // -0 and 0 are equal
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_bits(unsigned o) { return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o); }
__device__ __forceinline__ unsigned long long order_key(unsigned bits, int place) {
    return (unsigned long long)bits << 32 | (0xffffffffu - (unsigned)place);
}
__device__ __forceinline__ int place_of(unsigned long long key) { return (int)(0xffffffffu - (unsigned)key); }
// Sums relative to the maximum m, without the maximum's own term: d = sum e^(z - m) - 1, t = sum e^(z - m) (z - m);
// m = -inf: none.
struct Sums {
    float m;
    double d, t;
};
// The two taken together: the larger maximum stays, the other's terms and its 1 move to it.
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
    const Sums &hi = a.m >= b.m ? a : b, &lo = a.m >= b.m ? b : a;
    if (lo.m == -INFINITY) return hi;
    const double x = (double)lo.m - (double)hi.m, w = exp(x);
    Sums r;
    r.m = hi.m;
    r.d = hi.d + w * (1.0 + lo.d);
    r.t = hi.t + w * (lo.t + x * (1.0 + lo.d));
    return r;
}

// Shared memory of a CTA; the first CTA's is written by all of its cluster.
struct Shared {
    Sums part[kMaxCluster * kWarps];
    Sums total;
    int n_cand;
    unsigned long long cand[kSeg];        // candidates
    int segs[kMaxTop];
    unsigned least;
    unsigned seg_max[kMaxSegs];           // order_bits of the segments' maxima
};

__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(ptx::smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_remote(uint32_t a, unsigned v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t a, double v) {
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(a), "d"(v) : "memory");
}

// A lane's vectors of segment `seg`: virtual places seg * kSeg + (i * 32 + lane) * 4 + 0..3 of the row seen from the
// 16-byte boundary `head` logits in front of it; what lies outside the row is -inf.
__device__ __forceinline__ void load_segment(const float* row, int head, int vocab, int seg, float (&z)[4 * kVec]) {
    const int lane = threadIdx.x & 31;
    const int first = seg * kSeg - head;   // of the row
    if (first >= 0 && first + kSeg <= vocab) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(row + first) + i * 32 + lane);
            z[4 * i] = v.x;
            z[4 * i + 1] = v.y;
            z[4 * i + 2] = v.z;
            z[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4 * kVec; ++i) {
            const int v = first + ((i >> 2) * 32 + lane) * 4 + (i & 3);
            z[i] = v >= 0 && v < vocab ? __ldcg(row + v) : -INFINITY;
        }
    }
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2) k_logprobs(const LogprobArgs a) {
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.vocab;
    const int ctas = CLUSTER ? (int)(gridDim.x / a.rows) : 1, rank = CLUSTER ? (int)ptx::cluster_rank() : 0;
    const int r = CLUSTER ? blockIdx.x / ctas : blockIdx.x;
    ptx::griddep_wait();
    int token = 0;
    if (a.tokens) {
        token = a.tokens[r];
        if (token < 0 || token >= V) {   // the whole cluster leaves
            if (token >= V && rank == 0 && tid == 0) record_error(a.err, LLAMA_ERR_INVALID_ARG);
            return;
        }
    }
    if (CLUSTER) ptx::cluster_sync();   // every CTA of the cluster is there: the first one's shared memory is written from now on
    const float* row = a.logits + (size_t)r * V;
    const int head = (int)((uintptr_t)row >> 2 & 3);
    const int n_segs = (head + V + kSeg - 1) / kSeg;
    // ---------------------------------------------------------------- the pass: warp x of the row takes segments x, x + n, ...
    const int me = rank * kWarps + warp, all = ctas * kWarps;
    float m = -INFINITY, d = 0.f, t = 0.f;
    int bad = 0;
    float z[4 * kVec], next[4 * kVec];
    if (me < n_segs) load_segment(row, head, V, me, next);
    for (int seg = me; seg < n_segs; seg += all) {
#pragma unroll
        for (int i = 0; i < 4 * kVec; ++i) z[i] = next[i];
        if (seg + all < n_segs) load_segment(row, head, V, seg + all, next);
        float mx = z[0];
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 4 * kVec; ++i) {
            mx = fmaxf(mx, z[i]);
            odd |= !(z[i] < INFINITY);
        }
        bad |= odd;
        // the lane's running sums: d and t move to the new maximum
        const float mn = fmaxf(m, mx);
        if (mn != -INFINITY && !(mn == INFINITY)) {
            bool own = mn == m;   // the maximum's own term is outside already
            if (!own && m != -INFINITY) {
                const float x = m - mn, w = expf(x);   // x may be -inf: maxima of the type's ends
                t = w > 0.f ? w * fmaf(x, 1.f + d, t) : 0.f;
                d = w * (1.f + d);
            }
            float d4[4] = {0.f, 0.f, 0.f, 0.f}, t4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4 * kVec; ++i) {
                const float x = z[i] - mn;
                float e = expf(x);
                if (!own && x == 0.f) {   // the first of the maximum's places
                    own = true;
                    e = 0.f;
                }
                d4[i & 3] += e;
                if (e > 0.f) t4[i & 3] = fmaf(e, x, t4[i & 3]);
            }
            d += (d4[0] + d4[1]) + (d4[2] + d4[3]);
            t += (t4[0] + t4[1]) + (t4[2] + t4[3]);
            m = mn;
        }
        const unsigned best = __reduce_max_sync(0xffffffffu, order_bits(mx));
        if (a.n_top > 0 && lane == 0) {
            if (CLUSTER) st_remote(remote(&sh.seg_max[seg], 0), best);
            else sh.seg_max[seg] = best;
        }
    }
    Sums s{m, (double)d, (double)t};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Sums x;
        x.m = __shfl_xor_sync(0xffffffffu, s.m, o);
        x.d = __shfl_xor_sync(0xffffffffu, s.d, o);
        x.t = __shfl_xor_sync(0xffffffffu, s.t, o);
        // both lanes of a pair join in one order, so that all end with the same bits
        s = lane & o ? join(x, s) : join(s, x);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        Sums* to = &sh.part[me];
        if (CLUSTER) {
            st_remote(remote(&to->m, 0), __float_as_uint(s.m));
            st_remote(remote(&to->d, 0), s.d);
            st_remote(remote(&to->t, 0), bad ? (double)NAN : s.t);
        } else {
            *to = s;
            if (bad) to->t = NAN;
        }
    }
    if (CLUSTER) {
        ptx::cluster_sync();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    // ---------------------------------------------------------------- the row's sums (warp 0), the segments of the alternatives (the rest)
    if (warp == 0) {
        Sums x{-INFINITY, 0.0, 0.0};
        bool nan = false;
        for (int w = lane; w < all; w += 32) {
            const Sums y = sh.part[w];
            if (y.t != y.t) nan = true;
            else x = join(x, y);
        }
        nan = __any_sync(0xffffffffu, nan);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Sums y;
            y.m = __shfl_xor_sync(0xffffffffu, x.m, o);
            y.d = __shfl_xor_sync(0xffffffffu, x.d, o);
            y.t = __shfl_xor_sync(0xffffffffu, x.t, o);
            x = lane & o ? join(y, x) : join(x, y);
        }
        if (lane == 0) {
            // total: m, log(1 + d); NaN: a NaN or +inf in the row
            const double lse = nan ? (double)NAN : log1p(x.d);
            sh.total.m = x.m;
            sh.total.d = lse;
            const bool empty = x.m == -INFINITY && !nan;
            if (a.entropy) a.entropy[r] = empty ? 0.f : (float)(lse - x.t / (1.0 + x.d));
            if (a.logprobs) a.logprobs[r] = empty ? -INFINITY : (float)((double)(row[token] - x.m) - lse);
        }
    }
    if (a.n_top == 0) return;
    const int n = a.n_top, want = min(n, n_segs);
    if (tid == 0) sh.n_cand = 0;
    // the best `want` segments: a segment's rank is the number of better ones
    for (int g = tid; g < n_segs; g += kThreads) {
        const unsigned b = sh.seg_max[g];
        int better = 0;
        for (int x = 0; x < n_segs; ++x) {
            const unsigned o = sh.seg_max[x];
            better += o > b || (o == b && x < g);
        }
        if (better < want) sh.segs[better] = g;
        if (better == want - 1) sh.least = b;
    }
    __syncthreads();
    // their logits that may be among the n best: none below the least of the n segments' maxima (all, with fewer segments)
    const unsigned least = want < n ? 0u : sh.least;
    for (int k = warp; k < want; k += kWarps) {
        const int seg = sh.segs[k];
        float c[4 * kVec];
        load_segment(row, head, V, seg, c);
#pragma unroll
        for (int i = 0; i < 4 * kVec; ++i) {
            const int v = seg * kSeg - head + ((i >> 2) * 32 + lane) * 4 + (i & 3);
            const unsigned bits = order_bits(c[i]);
            if (v >= 0 && v < V && bits >= least) {
                const int at = atomicAdd(&sh.n_cand, 1);
                if (at < kSeg) sh.cand[at] = order_key(bits, v);
            }
        }
    }
    __syncthreads();
    const int found = sh.n_cand;
    auto put = [&](int k, unsigned long long key) {
        const float best = from_bits((unsigned)(key >> 32));
        const double lse = sh.total.d;
        a.top_ids[(size_t)r * n + k] = place_of(key);
        a.top_logprobs[(size_t)r * n + k] =
            sh.total.m == -INFINITY && lse == lse ? -INFINITY : (float)((double)(best - sh.total.m) - lse);
    };
    if (found <= kSeg) {
        for (int i = tid; i < found; i += kThreads) {
            const unsigned long long key = sh.cand[i];
            int better = 0;
            for (int x = 0; x < found; ++x) better += sh.cand[x] > key;
            if (better < n) put(better, key);
        }
        return;
    }
    // More candidates than the list holds (rows in order, rows of few values): a segment at a time, the n best kept in order
    // in the lanes of warp 0.
    unsigned long long mine = 0;
    for (int k = 0; k < want; ++k) {
        __syncthreads();
        const int v = sh.segs[k] * kSeg - head + tid;
        static_assert(kThreads == kSeg, "a logit a thread");
        sh.cand[tid] = v >= 0 && v < V ? order_key(order_bits(__ldcg(row + v)), v) : 0ull;
        __syncthreads();
        if (warp == 0)
            for (int i = 0; i < kSeg; ++i) {   // insertion: later ones move a lane on
                const unsigned long long key = sh.cand[i];
                const unsigned long long up = __shfl_up_sync(0xffffffffu, mine, 1);
                if (key > mine) mine = lane == 0 || up > key ? key : up;
            }
    }
    if (warp == 0 && lane < n) put(lane, mine);
}

}  // namespace
}  // namespace llama

using namespace llama;

extern "C" int llama_token_logprobs(const float* logits, int rows, int vocab, const int32_t* tokens, int n_top,
                                    float* logprobs, float* entropy, int32_t* top_ids, float* top_logprobs,
                                    int32_t* err_dev, void* stream) {
    if (rows < 0 || vocab <= 0 || vocab > (1 << 20) || n_top < 0 || n_top > kMaxTop || n_top > vocab)
        return LLAMA_ERR_INVALID_ARG;
    if ((tokens == nullptr) != (logprobs == nullptr)) return LLAMA_ERR_INVALID_ARG;
    if (rows == 0) return LLAMA_OK;
    if (!logits || (n_top > 0 && (!top_ids || !top_logprobs))) return LLAMA_ERR_INVALID_ARG;
    LogprobArgs a{logits, rows, vocab, n_top, tokens, logprobs, entropy, top_ids, top_logprobs, err_dev};
    cudaStream_t s = (cudaStream_t)stream;
    // CTAs per row: as many as the device has room for at once (two an SM), each with a segment per warp at least
    const int room = 2 * device_sm_count() / std::min(rows, 2 * device_sm_count());
    const int useful = ((vocab + kSeg - 1) / kSeg + kWarps - 1) / kWarps;
    int ctas = 1;
    while (2 * ctas <= std::min({room, useful, kMaxCluster})) ctas *= 2;
    const cudaError_t e = ctas == 1
                              ? launch_pdl(k_logprobs<false>, dim3(rows), dim3(kThreads), 0, s, a)
                              : launch_pdl_cluster(k_logprobs<true>, dim3(rows * ctas), dim3(kThreads), 0, ctas, s, a);
    return e == cudaSuccess ? LLAMA_OK : LLAMA_ERR_CUDA;
}
