// Beam search's selection: the best continuations of each request's beams.
//
// Candidate (k, v) of a request: beam k continued by token v, with the cumulative log
// probability  c(k, v) = score_k + z_kv - log sum_u e^{z_ku}.  A beam that has ended
// (its last token is the end token) stays as it is: its one candidate is (k, eos) at
// score_k.  The n_out largest candidates of a request's beams x vocab are wanted, in
// decreasing order, equal ones by increasing k * vocab + v.
//
// Within a row the order of candidates is the order of its logits (the row's score and
// normaliser shift all of them alike), so one pass over the logits gives everything:
// k_beam_scan reads a slice of a row once, keeps it in registers, and leaves the slice's
// maximum, its sum of exponentials and its n_out best (logit, token) pairs in order;
// k_beam_merge joins a request's slices.  Slice sums are fp32 (at most kSlice terms of at
// most 1); everything after them is fp64, since an fp32 cumulative score rounds different
// logits to equal candidates.
//
// Bound by the read of the logits.  Finding the best few must cost less than that: a bound
// on the n_out-th largest, from the threads' maxima, leaves a few dozen candidates per
// slice, which are ranked by counting the larger ones.  n_out rounds of a block-wide
// maximum instead took 179 us for 256 rows of 128,256 logits (n_out = 16).
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kPerThread = 32;                            // logits per thread
constexpr int kSlice = kScanThreads * kPerThread;
constexpr int kSplitsMax = (1 << 20) / kSlice;            // vocab <= 2^20
constexpr int kScanCap = 1024;                            // candidates ranked per slice
constexpr int kMergeThreads = 512;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMergeCap = 2048;                           // candidates ranked per request
constexpr int kBeamsMax = 32;
constexpr int kOutMax = 64;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

// Logits in an order-preserving unsigned form (every number, -inf included, above 0).
// Adding +0 makes the two zeros one value.
__device__ __forceinline__ unsigned ordered(float f) {
    const unsigned u = __float_as_uint(__fadd_rn(f, 0.f));
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(unsigned o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ unsigned long long ordered(double f) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(__dadd_rn(f, 0.));
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// A slice's candidate: the logit's ordered form above the complement of its token, so
// that a larger key is a better candidate (equal logits: the lower token).  0: none.
__device__ __forceinline__ unsigned long long cand_key(float z, int v) {
    return ((unsigned long long)ordered(z) << 32) | (unsigned)~v;
}

struct BeamArgs {
    const float* logits;
    const float* scores;
    const int* last;
    int eos;
    int beams, vocab, n_out, splits;
    float2* part;                 // [rows][splits]: slice maximum, sum of e^(z - maximum)
    unsigned long long* cand;     // [rows][splits][n_out] candidate keys, decreasing
    int* parents;
    int* tokens;
    float* best;
};

// A beam whose candidates its logits decide (the others are not read).
__device__ __forceinline__ bool row_ended(const BeamArgs& a, int row) { return a.last && __ldcg(a.last + row) == a.eos; }
__device__ __forceinline__ bool row_live(const BeamArgs& a, int row) {
    return __ldcg(a.scores + row) != -INFINITY && !row_ended(a, row);
}

__device__ __forceinline__ unsigned long long warp_max(unsigned long long k) {
    const unsigned hi = __reduce_max_sync(kAll, (unsigned)(k >> 32));
    const unsigned lo = __reduce_max_sync(kAll, (unsigned)(k >> 32) == hi ? (unsigned)k : 0u);
    return ((unsigned long long)hi << 32) | lo;
}

// The q-th largest of the lanes' keys (equal keys counted one by one), q <= 32.
template <typename K>
__device__ __forceinline__ K warp_nth(K key, int q) {
    const int lane = threadIdx.x & 31;
    K top{};
    for (int i = 0; i < q; ++i) {
        if constexpr (sizeof(K) == 8) top = warp_max(key);
        else top = __reduce_max_sync(kAll, key);
        const unsigned who = __ballot_sync(kAll, key == top);
        if (lane == __ffs(who) - 1) key = 0;
    }
    return top;
}

// 2^x on the special-function unit (ex2.approx.ftz: relative error 2^-22).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// VEC: rows of whole 16-byte vectors, read as such; a thread then holds runs of four.
template <bool VEC>
__global__ void __launch_bounds__(kScanThreads, 4) k_beam_scan(const BeamArgs a) {
    __shared__ unsigned s_max[kScanWarps], s_nth[kScanWarps];
    __shared__ float s_sum[kScanWarps];
    __shared__ unsigned long long s_list[kScanCap];
    __shared__ unsigned long long s_key[kScanWarps];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.y, split = blockIdx.x;
    ptx::griddep_wait();
    if (tid == 0) ptx::griddep_launch_dependents();   // the merge waits for this grid before it reads
    if (!row_live(a, row)) return;
    const float* z = a.logits + (size_t)row * a.vocab;
    const int v0 = split * kSlice, n = min(kSlice, a.vocab - v0);
    auto at = [&](int i) { return VEC ? (i >> 2) * (4 * kScanThreads) + tid * 4 + (i & 3) : tid + i * kScanThreads; };
    float x[kPerThread];
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kPerThread; i += 4) {
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (at(i) < n) v = __ldcg(reinterpret_cast<const float4*>(z + v0 + at(i)));
            x[i] = v.x;
            x[i + 1] = v.y;
            x[i + 2] = v.z;
            x[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) x[i] = at(i) < n ? __ldcg(z + v0 + at(i)) : -INFINITY;
    }
    float most = x[0];
#pragma unroll
    for (int i = 1; i < kPerThread; ++i) most = fmaxf(most, x[i]);
    // A lower bound of the slice's n_out-th largest logit: in every warp at least
    // ceil(n_out / kScanWarps) threads have a logit of the warp's bound or more, so the
    // smallest of the warps' bounds has n_out logits at or above it -- and, a thread in
    // kScanWarps holding one of them, not many more.
    const unsigned mine = at(0) < n ? ordered(most) : 0u;
    const unsigned wmax = __reduce_max_sync(kAll, mine);
    const unsigned nth = warp_nth(mine, (a.n_out + kScanWarps - 1) / kScanWarps);
    if (lane == 0) {
        s_max[warp] = wmax;
        s_nth[warp] = nth;
    }
    if (tid == 0) s_n = 0;
    __syncthreads();
    unsigned top_key = 0, bound = 0xffffffffu;
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) {
        top_key = max(top_key, s_max[w]);
        bound = min(bound, s_nth[w]);
    }
    // every logit at or above the bound goes to the list
    if (mine >= bound) {
#pragma unroll
        for (int i = 0; i < kPerThread; ++i)
            if (at(i) < n && ordered(x[i]) >= bound) {
                const int p = atomicAdd(&s_n, 1);
                if (p < kScanCap) s_list[p] = cand_key(x[i], v0 + at(i));
            }
    }
    const float m = unordered(top_key);
    const float top = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) sum += ex2((x[i] - top) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    const size_t slot = (size_t)row * a.splits + split;
    unsigned long long* out = a.cand + slot * a.n_out;
    if (tid == 0) {
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) sum += s_sum[w];
        a.part[slot] = make_float2(m, sum);
    }
    const int found = s_n;
    if (found <= kScanCap) {
        // keys differ, so a key's place is the number of larger ones
        for (int c = tid; c < found; c += kScanThreads) {
            const unsigned long long k = s_list[c];
            int rank = 0;
            for (int i = 0; i < found; ++i) rank += s_list[i] > k;
            if (rank < a.n_out) out[rank] = k;
        }
        for (int c = found + tid; c < a.n_out; c += kScanThreads) out[c] = 0;
        return;
    }
    // Many equal logits (a mask, say): n_out rounds in which the best remaining
    // candidate leaves and its thread finds its next one.
    unsigned long long best = ~0ull, own = ~0ull;
    for (int o = 0; o < a.n_out; ++o) {
        if (own == best) {   // the first round: every thread
            own = 0;
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) {
                const unsigned long long k = cand_key(x[i], v0 + at(i));
                if (at(i) < n && k < best) own = max(own, k);
            }
        }
        best = warp_max(own);
        __syncthreads();   // the keys of the round before were read
        if (lane == 0) s_key[warp] = best;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) best = max(best, s_key[w]);
        if (tid == 0) out[o] = best;
    }
}

// A candidate of the merge: decreasing value, then increasing place.
struct Cand {
    unsigned long long value;   // ordered form; 0: none
    unsigned place;             // beam * vocab + token
};
__device__ __forceinline__ bool better(const Cand& p, const Cand& q) {
    return p.value > q.value || (p.value == q.value && p.place < q.place);
}
__device__ __forceinline__ Cand warp_best(Cand c) {
    const unsigned hi = __reduce_max_sync(kAll, (unsigned)(c.value >> 32));
    const unsigned lo = __reduce_max_sync(kAll, (unsigned)(c.value >> 32) == hi ? (unsigned)c.value : 0u);
    const unsigned long long v = ((unsigned long long)hi << 32) | lo;
    const unsigned place = __reduce_min_sync(kAll, c.value == v ? c.place : 0xffffffffu);
    return {v, place};
}

// One CTA per request.  The scan's idea once more, on the beams x slices lists: the
// bound comes from the lists' d-th keys (d = 1 unless there are fewer lists than
// wanted candidates), the keys at or above it are gathered and ranked by counting.
__global__ void __launch_bounds__(kMergeThreads) k_beam_merge(const BeamArgs a) {
    // a live beam's largest logit, and its score - log sum e^(z - largest): kept apart, since
    // next to a mask of the type's lowest value a score would be lost
    __shared__ float s_top[kBeamsMax];
    __shared__ double s_shift[kBeamsMax];
    __shared__ int s_mode[kBeamsMax];       // 0: live, 1: ended, 2: at -inf
    __shared__ unsigned long long s_nth[kMergeWarps];
    __shared__ unsigned long long s_value[kMergeCap];
    __shared__ unsigned s_place[kMergeCap];
    __shared__ Cand s_best[kMergeWarps];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.x;
    const int row0 = g * a.beams;
    ptx::griddep_wait();
    if (tid == 0) s_n = 0;
    // normalisers: one warp per beam
    for (int k = warp; k < a.beams; k += kMergeWarps) {
        const int row = row0 + k;
        const float score = __ldcg(a.scores + row);
        if (lane == 0) {
            s_mode[k] = score == -INFINITY ? 2 : row_ended(a, row) ? 1 : 0;
            s_top[k] = 0.f;
            s_shift[k] = score;
        }
        if (!row_live(a, row)) continue;
        const float2* p = a.part + (size_t)row * a.splits;
        float2 ms[kSplitsMax / 32];
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kSplitsMax / 32; ++i) {
            const int s = lane + 32 * i;
            ms[i] = s < a.splits ? __ldcg(p + s) : make_float2(-INFINITY, 0.f);
            m = fmaxf(m, ms[i].x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        if (m == -INFINITY) continue;   // no token has a probability: every candidate is at -inf
        double sum = 0;
#pragma unroll
        for (int i = 0; i < kSplitsMax / 32; ++i) sum += (double)(ms[i].y * ex2((ms[i].x - m) * kLog2e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (lane == 0) {
            s_top[k] = m;
            s_shift[k] = (double)score - log(sum);
        }
    }
    __syncthreads();
    const int lists = a.beams * a.splits;
    auto fetch = [&](int list, int pos) -> Cand {
        const int k = list / a.splits, s = list - k * a.splits;
        const unsigned base = (unsigned)k * a.vocab;
        if (s_mode[k] != 0) {
            if (s != 0) return {0ull, 0xffffffffu};
            if (s_mode[k] == 1) {
                // (k, eos) first, then the tokens that do not follow an end, at -inf
                if (pos == 0) return {ordered(s_shift[k]), base + a.eos};
                const int v = pos - 1 < a.eos ? pos - 1 : pos;
                return {ordered((double)-INFINITY), base + v};
            }
            return {ordered((double)-INFINITY), base + pos};
        }
        const unsigned long long key = __ldcg(a.cand + ((size_t)(row0 + k) * a.splits + s) * a.n_out + pos);
        if (key == 0) return {0ull, 0xffffffffu};
        const double below = (double)unordered((unsigned)(key >> 32)) - (double)s_top[k];
        return {ordered(below + s_shift[k]), base + ~(unsigned)key};
    };
    // list i belongs to warp i % kMergeWarps: at least `each` lists per warp
    const int q = (a.n_out + kMergeWarps - 1) / kMergeWarps, each = lists / kMergeWarps;
    const int d = each == 0 ? 1 : min(a.n_out, (q + min(each, 32) - 1) / min(each, 32));
    unsigned long long mine = 0;
    for (int i = lane * kMergeWarps + warp; i < lists; i += kMergeThreads) mine = max(mine, fetch(i, d - 1).value);
    mine = warp_nth(mine, (q + d - 1) / d);
    if (lane == 0) s_nth[warp] = mine;
    __syncthreads();
    unsigned long long bound = ~0ull;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) bound = min(bound, s_nth[w]);
    // Candidates at -inf count only where the others are fewer than n_out (a first step's
    // idle beams hold most of the lists' heads at -inf or empty, and so the bound down).
    const int total = lists * a.n_out;
    const unsigned long long lowest = ordered((double)-INFINITY);
    bound = max(bound, lowest + 1);
    int found;
    while (true) {
#pragma unroll 4
        for (int i = tid; i < total; i += kMergeThreads) {
            const int list = i / a.n_out;
            const Cand c = fetch(list, i - list * a.n_out);
            if (c.value >= bound) {
                const int p = atomicAdd(&s_n, 1);
                if (p < kMergeCap) {
                    s_value[p] = c.value;
                    s_place[p] = c.place;
                }
            }
        }
        __syncthreads();
        found = s_n;
        if (found >= a.n_out || bound == lowest) break;
        __syncthreads();   // everyone has read the count
        if (tid == 0) s_n = 0;
        __syncthreads();
        bound = lowest;
    }
    auto emit = [&](int o, const Cand& c) {
        const size_t at = (size_t)g * a.n_out + o;
        a.parents[at] = row0 + (int)(c.place / (unsigned)a.vocab);
        a.tokens[at] = (int)(c.place % (unsigned)a.vocab);
        a.best[at] = (float)__longlong_as_double(
            (long long)(c.value >> 63 ? c.value & 0x7fffffffffffffffull : ~c.value));
    };
    if (found <= kMergeCap) {
        for (int c = tid; c < found; c += kMergeThreads) {
            const Cand x{s_value[c], s_place[c]};
            int rank = 0;
            for (int i = 0; i < found; ++i) rank += better(Cand{s_value[i], s_place[i]}, x);
            if (rank < a.n_out) emit(rank, x);
        }
        return;
    }
    // many equal candidates: n_out rounds over all keys below the last one taken
    Cand last{~0ull, 0u};
    for (int o = 0; o < a.n_out; ++o) {
        Cand best{0ull, 0xffffffffu};
        for (int i = tid; i < total; i += kMergeThreads) {
            const int list = i / a.n_out;
            const Cand c = fetch(list, i - list * a.n_out);
            if (better(last, c) && better(c, best)) best = c;
        }
        best = warp_best(best);
        __syncthreads();
        if (lane == 0) s_best[warp] = best;
        __syncthreads();
        last = warp_best(lane < kMergeWarps ? s_best[lane] : Cand{0ull, 0xffffffffu});
        if (tid == 0) emit(o, last);
    }
}

int beam_splits(int vocab) { return (vocab + kSlice - 1) / kSlice; }
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

bool beam_dims_ok(int groups, int beams, int vocab, int n_out) {
    return groups >= 0 && beams >= 1 && beams <= kBeamsMax && vocab >= 1 && vocab <= (1 << 20) && n_out >= 1 &&
           n_out <= kOutMax && n_out <= vocab && (long long)groups * beams <= 65535;
}

}  // namespace
}  // namespace llama

using namespace llama;

extern "C" size_t llama_beam_select_workspace_bytes(int groups, int beams, int vocab, int n_out) {
    if (groups <= 0 || !beam_dims_ok(groups, beams, vocab, n_out)) return 0;
    const size_t lists = (size_t)groups * beams * beam_splits(vocab);
    return align256(lists * sizeof(float2)) + align256(lists * n_out * sizeof(unsigned long long));
}

extern "C" int llama_beam_select(const float* logits, int groups, int beams, int vocab, const float* scores,
                                 const int32_t* last, int eos, int n_out, int32_t* parents, int32_t* tokens,
                                 float* out_scores, void* ws, size_t ws_bytes, void* stream) {
    if (!beam_dims_ok(groups, beams, vocab, n_out)) return LLAMA_ERR_INVALID_ARG;
    if (last && (eos < 0 || eos >= vocab)) return LLAMA_ERR_INVALID_ARG;
    if (groups == 0) return LLAMA_OK;
    if (!logits || !scores || !parents || !tokens || !out_scores) return LLAMA_ERR_INVALID_ARG;
    if (!ws || ws_bytes < llama_beam_select_workspace_bytes(groups, beams, vocab, n_out)) return LLAMA_ERR_WORKSPACE;
    if ((uintptr_t)ws & 15) return LLAMA_ERR_INVALID_ARG;
    BeamArgs a{};
    a.logits = logits;
    a.scores = scores;
    a.last = last;
    a.eos = eos;
    a.beams = beams;
    a.vocab = vocab;
    a.n_out = n_out;
    a.splits = beam_splits(vocab);
    a.part = (float2*)ws;
    a.cand = (unsigned long long*)((uint8_t*)ws + align256((size_t)groups * beams * a.splits * sizeof(float2)));
    a.parents = parents;
    a.tokens = tokens;
    a.best = out_scores;
    cudaStream_t s = (cudaStream_t)stream;
    const bool vec = vocab % 4 == 0 && ((uintptr_t)logits & 15) == 0;
    if (launch_pdl(vec ? k_beam_scan<true> : k_beam_scan<false>, dim3(a.splits, groups * beams), dim3(kScanThreads), 0, s,
                   a) != cudaSuccess)
        return LLAMA_ERR_CUDA;
    if (launch_pdl(k_beam_merge, dim3(groups), dim3(kMergeThreads), 0, s, a) != cudaSuccess) return LLAMA_ERR_CUDA;
    return LLAMA_OK;
}
