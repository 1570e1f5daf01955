// llama_token_logprobs: log probabilities of given tokens, entropy and top alternatives of fp32 logits.
//
// With m = max z = z_u (u the first such token) and e_v = e^(z_v - m), d = sum_{v != u} e_v and
// t = sum e_v (z_v - m) (terms of weight 0 left out):
//   log p_v = (z_v - m) - log(1 + d),   H = log(1 + d) - t / (1 + d),
// all without cancellation: the terms of t are <= 0, and leaving the 1 out of the sums keeps small d.
//
// One pass over the logits.  A row is cut into segments of kSeg logits; a warp takes a segment at a time, all its
// loads issued ahead, and keeps its running maximum, the lanes' parts of d and t relative to it (the maximum's own term
// left out), and the maximum of each segment.  (A maximum per lane moves in most segments for some lane of the warp, the warp's
// a few times a row: 23 instructions a logit against 9.)  The warps' triples are joined in a tree, in fp32 (in fp64 that
// took 40 us a row).
// The n largest logits lie in the n segments with
// the largest maxima (equal maxima: the first segments): a segment outside has n segments whose best is better than all
// it has.  So the alternatives come from n segments read a second time, from L2.
//
// Few rows are split over a cluster of CTAs of 16 warps (their triples and segment maxima in distributed shared memory,
// the first CTA finishes the row).  Many rows (kManyRows per SM or more) take a CTA of 4 warps each, 7 to an SM (72
// registers): one finishes its row while the others read, and no round of large CTAs ends half empty (924 rows of 128256
// logits: 137 us with 16 warps a row, 75 so: 6.3 TB/s, 0.95 of the copy rate).  Few rows are bound by a chain of round
// trips: 1 row with 20 alternatives 9.9 us, 32 rows with 5 11.7.  In between, with 5 alternatives: 64 rows 15 us, 128 21,
// 152 22; from 153 on a row has one CTA of 16 warps, 27 (153) to 32 (304), and from 305 on a second round of them, 43 (305)
// to 59 (607); 608 in small CTAs 57, 1024 83.  (305 rows are 156 MB, 23 us: the worst place of the rule.)
#include <algorithm>
#include <climits>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int kMaxTop = 32;
constexpr int kFewThreads = 512, kManyThreads = 128;
constexpr int kManyRows = 4;
constexpr int kVec = 4;                        // 16-byte vectors of a lane in a segment
constexpr int kSeg = 32 * 4 * kVec;            // 512 logits
constexpr int kMaxSegs = (1 << 20) / kSeg + 1; // of a row (one more where it starts off 16 bytes)
constexpr int kMaxCluster = 8;
// Logits of a short row that are all ranked, each by a look at all others (1024 rows of 500 logits all ranked 50 us, the
// candidates narrowed 10.5; 1 row of 250: 7.2 and 8.8; 1024 rows of 170: 11.5 and 10.1).  At least 4 * 32 + 3: with more
// logits every lane of the row's first segment has one, and 32 lanes with a logit bound 32 alternatives (of the last segment
// most lanes may have none).
constexpr int kListedFew = 256, kListedMany = 160;

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
// m = -inf: none.  A NaN in d stays: a row with a NaN or +inf.
struct Sums {
    float m, d, t;
};
// e^x, x <= 0: 2^-22 relative beside the rounding of x log2 e; 0 below 2^-126.
__device__ __forceinline__ float exp_neg(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}
// The larger, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
constexpr float kFar = -200.f;   // e^kFar is 0: nothing below it (or -inf) is told apart, and 0 * -inf does not arise
// The two taken together: the larger maximum stays, the other's terms and its 1 move to it.
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
    const bool first = a.m >= b.m;
    const float hm = first ? a.m : b.m, hd = first ? a.d : b.d, ht = first ? a.t : b.t;
    const float lm = first ? b.m : a.m, ld = first ? b.d : a.d, lt = first ? b.t : a.t;
    const float x = fmaxf(lm - hm, kFar), w = lm == -INFINITY ? 0.f : exp_neg(x), one = 1.f + ld;
    return Sums{hm, __fmaf_rn(w, one, hd), __fmaf_rn(w, __fmaf_rn(x, one, lt), ht)};
}
__device__ __forceinline__ Sums join_warp(Sums s) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Sums x;
        x.m = __shfl_xor_sync(0xffffffffu, s.m, o);
        x.d = __shfl_xor_sync(0xffffffffu, s.d, o);
        x.t = __shfl_xor_sync(0xffffffffu, s.t, o);
        // both lanes of a pair join in one order, so that all end with the same bits
        s = lane & o ? join(x, s) : join(s, x);
    }
    return s;
}
__device__ __forceinline__ float add_warp(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Shared memory of a CTA; the first CTA's is written by all of its cluster.
struct Shared {
    Sums part[kMaxCluster * kFewThreads / 32];
    Sums total;                           // m, log(1 + d), -
    int n_cand;
    unsigned long long cand[kMaxTop * 32];   // candidates; the lanes' best of the segments
    int tally[2][kFewThreads / 32];
    int segs[kMaxTop];
    unsigned least;
    alignas(16) unsigned seg_max[kMaxSegs + 3];   // order_bits of the segments' maxima, and zeros up to a multiple of 4
};

__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(ptx::smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_remote(uint32_t a, unsigned v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
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

// The n-th largest of the lanes' bests, the best of each lane's 16 logits of the segments sh.segs[0 .. want - 1], found by
// halving the keys' range.  A function of its own: seldom called, and within the kernel its instructions cost every row 0.6 us.
template <int kThreads>
__device__ __noinline__ unsigned long long nth_of_lanes(Shared& sh, const float* row, int head, int V, int want, int n) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int k = warp; k < want; k += kWarps) {
        const int seg = sh.segs[k];
        float c[4 * kVec];
        load_segment(row, head, V, seg, c);
        unsigned best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < 4 * kVec; ++i) {   // by increasing place
            const int v = seg * kSeg - head + ((i >> 2) * 32 + lane) * 4 + (i & 3);
            const unsigned bits = order_bits(c[i]);
            if (v >= 0 && v < V && bits > best) {
                best = bits;
                at = v;
            }
        }
        sh.cand[k * 32 + lane] = best ? order_key(best, at) : 0ull;
    }
    __syncthreads();
    unsigned long long least = 0;
    for (int bit = 63, turn = 0; bit >= 0; --bit, turn ^= 1) {
        if (bit == 31) {   // the places: all below 2^20
            bit = 19;
            least |= 0xfff00000u;
        }
        const unsigned long long above = least | 1ull << bit;
        int reach = 0;
        for (int i = tid; i < want * 32; i += kThreads) reach += sh.cand[i] >= above;
        reach = __reduce_add_sync(0xffffffffu, reach);
        if (lane == 0) sh.tally[turn][warp] = reach;
        __syncthreads();
        reach = 0;
        for (int w = 0; w < kWarps; ++w) reach += sh.tally[turn][w];
        if (reach >= n) least = above;
        if (reach == n) break;
    }
    __syncthreads();
    return least;
}

template <int kThreads, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, kThreads == kManyThreads ? 7 : 2) k_logprobs(const LogprobArgs a) {
    constexpr int kWarps = kThreads / 32;
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
    if (rank == 0 && tid < 3) sh.seg_max[n_segs + tid] = 0;
    // ---------------------------------------------------------------- the pass: warp x of the row takes segments x, x + n, ...
    const int me = rank * kWarps + warp, all = ctas * kWarps;
    const unsigned none = order_bits(-INFINITY);
    unsigned top = none;             // the warp's maximum so far
    float m = -INFINITY, d = 0.f, t = 0.f;   // d, t: this lane's part
    auto take = [&](int seg, float (&z)[4 * kVec]) {
        float mx = z[0];
#pragma unroll
        for (int i = 1; i < 4 * kVec; ++i) mx = fmaxf(mx, z[i]);
        const unsigned bits = order_bits(mx), best = __reduce_max_sync(0xffffffffu, bits);
        if (a.n_top > 0 && lane == 0) {
            if (CLUSTER) st_remote(remote(&sh.seg_max[seg], 0), best);
            else sh.seg_max[seg] = best;
        }
        if (best > top) {   // the sums move to the new maximum, whose first place is left out of them
            const float mn = from_bits(best), x = fmaxf(m - mn, kFar), w = top == none ? 0.f : exp_neg(x);
            const float own = lane == 0 ? 1.f + d : d;   // lane 0 takes the old maximum's term in
            t = w * __fmaf_rn(x, own, t);
            d = w * own;
            m = mn;
            top = best;
            if (lane == __ffs(__ballot_sync(0xffffffffu, bits == best)) - 1) {
                bool out = false;
#pragma unroll
                for (int i = 0; i < 4 * kVec; ++i)
                    if (!out && z[i] == mn) {
                        out = true;
                        z[i] = -INFINITY;
                    }
            }
            if (mn == INFINITY) d = NAN;
        }
        if (top == none) {   // nothing above -inf so far; a NaN among it stays
#pragma unroll
            for (int i = 0; i < 4 * kVec; ++i)
                if (z[i] != z[i]) d = NAN;
            return;
        }
        float d4[4] = {0.f, 0.f, 0.f, 0.f}, t4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4 * kVec; ++i) {
            const float x = max_nan(z[i] - m, kFar), e = exp_neg(x);
            d4[i & 3] += e;
            t4[i & 3] = __fmaf_rn(e, x, t4[i & 3]);
        }
        d += (d4[0] + d4[1]) + (d4[2] + d4[3]);
        t += (t4[0] + t4[1]) + (t4[2] + t4[3]);
    };
    // a segment's loads go out before the one in front of it is taken
    float z0[4 * kVec], z1[4 * kVec];
    int seg = me;
    if (seg < n_segs) load_segment(row, head, V, seg, z0);
    while (seg < n_segs) {
        if (seg + all < n_segs) load_segment(row, head, V, seg + all, z1);
        take(seg, z0);
        seg += all;
        if (seg >= n_segs) break;
        if (seg + all < n_segs) load_segment(row, head, V, seg + all, z0);
        take(seg, z1);
        seg += all;
    }
    const Sums s{m, add_warp(d), add_warp(t)};
    if (lane == 0) {
        Sums* to = &sh.part[me];
        if (CLUSTER) {
            st_remote(remote(&to->m, 0), __float_as_uint(s.m));
            st_remote(remote(&to->d, 0), __float_as_uint(s.d));
            st_remote(remote(&to->t, 0), __float_as_uint(s.t));
        } else {
            *to = s;
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
        Sums x{-INFINITY, 0.f, 0.f};
        for (int w = lane; w < all; w += 32) x = join(x, sh.part[w]);
        x = join_warp(x);
        if (lane == 0) {
            const bool empty = x.m == -INFINITY && x.d == x.d;
            const float lse = x.d == x.d ? log1pf(x.d) : NAN;
            sh.total = Sums{x.m, lse, 0.f};
            if (a.entropy) a.entropy[r] = empty ? 0.f : lse - x.t / (1.f + x.d);
            if (a.logprobs) a.logprobs[r] = empty ? -INFINITY : (row[token] - x.m) - lse;
        }
    }
    if (a.n_top == 0) return;
    const int n = a.n_top, want = min(n, n_segs);
    if (tid == 0) sh.n_cand = 0;
    // the best `want` segments
    if constexpr (kThreads == kManyThreads) {
        // one warp, a segment a round (the other CTAs of the SM have the schedulers): lane x holds the best of segments x,
        // x + 32, ... that are left, equal ones by increasing segment
        if (warp == 1) {
            unsigned b = 0;
            int at = INT_MAX;
            auto look = [&] {
                b = 0;
                for (int g = lane; g < n_segs; g += 32) {
                    const unsigned o = sh.seg_max[g];
                    if (o > b) {
                        b = o;
                        at = g;
                    }
                }
            };
            look();
            for (int k = 0; k < want; ++k) {
                const unsigned best = __reduce_max_sync(0xffffffffu, b);
                const int seg = __reduce_min_sync(0xffffffffu, b == best ? at : INT_MAX);
                if (lane == 0) {
                    sh.segs[k] = seg;
                    sh.least = best;
                }
                if (k + 1 < want && (seg & 31) == lane) {
                    sh.seg_max[seg] = 0;   // below every logit's bits
                    look();
                }
                __syncwarp();
            }
        }
    } else {
        // all threads: a segment's rank is the number of better ones, those of the same best in front among them.  Four
        // at a time: the loop takes the latency of its reads, and a third of a row's time one by one (15.1 us, here
        // 9.9; 1 row, 20 alternatives).
        const int n4 = (n_segs + 3) & ~3;
        const uint4* seg4 = reinterpret_cast<const uint4*>(sh.seg_max);
        for (int g0 = warp * 32; g0 < n_segs; g0 += kThreads) {
            const int g = g0 + lane;
            const unsigned b = g < n_segs ? sh.seg_max[g] : 0;
            int better = 0;
#pragma unroll 1
            for (int after = 0; after < 2; ++after) {   // the segments in front of the warp's 32, and behind them
                const unsigned least = b + after;
#pragma unroll 4
                for (int x = after ? g0 / 4 + 8 : 0; x < (after ? n4 : g0) / 4; ++x) {
                    const uint4 o = seg4[x];
                    better += (o.x >= least) + (o.y >= least) + (o.z >= least) + (o.w >= least);
                }
            }
#pragma unroll 8
            for (int x = 0; x < 32; ++x) better += __shfl_sync(0xffffffffu, b, x) >= b + (x >= lane);
            if (g >= n_segs) continue;
            if (better < want) sh.segs[better] = g;
            if (better == want - 1) sh.least = b;
        }
    }
    __syncthreads();
    // Their logits that may be among the n best are listed: none is below the least of the n segments' maxima (of fewer
    // segments all may).  Where these are more than the list holds (rows in order, rows of few values), or all of a row that is
    // not short: the n-th largest of the lanes' bests bounds the n best logits, n lanes reach it, and so at most 16 n <= kSeg
    // logits.  (One warp that sorted the segments in took 108 us for rows of 4584 logits, 20 alternatives; so 11.4.)
    unsigned long long least = want < n ? 0ull : (unsigned long long)sh.least << 32;
    bool narrow = want < n && V > (kThreads == kManyThreads ? kListedMany : kListedFew);
    while (true) {
        if (narrow) least = nth_of_lanes<kThreads>(sh, row, head, V, want, n);
        for (int k = warp; k < want; k += kWarps) {
            const int seg = sh.segs[k];
            float c[4 * kVec];
            load_segment(row, head, V, seg, c);
#pragma unroll
            for (int i = 0; i < 4 * kVec; ++i) {
                const int v = seg * kSeg - head + ((i >> 2) * 32 + lane) * 4 + (i & 3);
                const unsigned bits = order_bits(c[i]);
                if (v >= 0 && v < V && order_key(bits, v) >= least) {
                    const int at = atomicAdd(&sh.n_cand, 1);
                    if (at < kSeg) sh.cand[at] = order_key(bits, v);
                }
            }
        }
        __syncthreads();
        if (narrow || sh.n_cand <= kSeg) break;
        narrow = true;
        __syncthreads();
        if (tid == 0) sh.n_cand = 0;
    }
    // a candidate's place is the number of better ones
    const int found = sh.n_cand;
    const float lse = sh.total.d;
    for (int i = tid; i < found; i += kThreads) {
        const unsigned long long key = sh.cand[i];
        int better = 0;
        for (int x = 0; x < found; ++x) better += sh.cand[x] > key;
        if (better < n) {
            const float best = from_bits((unsigned)(key >> 32));
            a.top_ids[(size_t)r * n + better] = place_of(key);
            a.top_logprobs[(size_t)r * n + better] =
                sh.total.m == -INFINITY && lse == lse ? -INFINITY : (best - sh.total.m) - lse;
        }
    }
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
    const int n_sm = device_sm_count();
    cudaError_t e;
    if (rows >= kManyRows * n_sm) {
        e = launch_pdl(k_logprobs<kManyThreads, false>, dim3(rows), dim3(kManyThreads), 0, s, a);
    } else {
        // CTAs per row: as many as the device has room for at once (two an SM), each with a segment per warp at least
        const int room = 2 * n_sm / std::min(rows, 2 * n_sm);
        const int useful = ((vocab + kSeg - 1) / kSeg + kFewThreads / 32 - 1) / (kFewThreads / 32);
        int ctas = 1;
        while (2 * ctas <= std::min({room, useful, kMaxCluster})) ctas *= 2;
        e = ctas == 1 ? launch_pdl(k_logprobs<kFewThreads, false>, dim3(rows), dim3(kFewThreads), 0, s, a)
                      : launch_pdl_cluster(k_logprobs<kFewThreads, true>, dim3(rows * ctas), dim3(kFewThreads), 0, ctas, s, a);
    }
    return e == cudaSuccess ? LLAMA_OK : LLAMA_ERR_CUDA;
}
