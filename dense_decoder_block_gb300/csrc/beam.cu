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
// k_beam_merge joins a request's slices: normalisers in 64 bits from the slices' (m, s),
// then n_out rounds of a tournament over the heads of the beams x slices sorted lists,
// candidates compared by their 64-bit value and then by place.  Slice sums are fp32
// (at most kSlice terms of at most 1, relative error below 1e-6); everything after them
// is fp64, since an fp32 cumulative score rounds different logits to equal candidates.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kPerThread = 32;                            // logits per thread
constexpr int kSlice = kScanThreads * kPerThread;
constexpr int kMergeThreads = 512;
constexpr int kMergeWarps = kMergeThreads / 32;
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

__global__ void __launch_bounds__(kScanThreads) k_beam_scan(const BeamArgs a) {
    __shared__ unsigned long long s_key[kScanWarps];
    __shared__ float s_sum[kScanWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.y, split = blockIdx.x;
    ptx::griddep_wait();
    if (tid == 0) ptx::griddep_launch_dependents();   // the merge waits for this grid before it reads
    if (!row_live(a, row)) return;
    const float* z = a.logits + (size_t)row * a.vocab;
    const int v0 = split * kSlice, n = min(kSlice, a.vocab - v0);
    float x[kPerThread];
    unsigned long long mine = 0;   // this thread's best remaining candidate
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int j = tid + i * kScanThreads;
        x[i] = j < n ? __ldcg(z + v0 + j) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int j = tid + i * kScanThreads;
        if (j < n) mine = max(mine, cand_key(x[i], v0 + j));
    }
    // the slice's maximum is its best candidate's logit
    unsigned long long best = warp_max(mine);
    if (lane == 0) s_key[warp] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) best = max(best, s_key[w]);
    const float m = unordered((unsigned)(best >> 32));
    const float top = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) sum += exp2f((x[i] - top) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    const size_t slot = (size_t)row * a.splits + split;
    if (tid == 0) {
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) sum += s_sum[w];
        a.part[slot] = make_float2(m, sum);
    }
    // n_out rounds: the best remaining candidate leaves, its thread finds its next one
    for (int o = 0; o < a.n_out; ++o) {
        if (tid == 0) a.cand[slot * a.n_out + o] = best;
        if (best != 0 && mine == best) {
            mine = 0;
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) {
                const int j = tid + i * kScanThreads;
                const unsigned long long k = cand_key(x[i], v0 + j);
                if (j < n && k < best) mine = max(mine, k);
            }
        }
        best = warp_max(mine);
        __syncthreads();   // the keys of the round before were read
        if (lane == 0) s_key[warp] = best;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) best = max(best, s_key[w]);
    }
}

// A candidate in the tournament: decreasing value, then increasing place.
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

__global__ void __launch_bounds__(kMergeThreads) k_beam_merge(const BeamArgs a) {
    // a live beam's largest logit, and its score - log sum e^(z - largest): kept apart, since
    // next to a mask of the type's lowest value a score would be lost
    __shared__ float s_top[kBeamsMax];
    __shared__ double s_shift[kBeamsMax];
    __shared__ Cand s_best[kMergeWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.x;
    const int row0 = g * a.beams;
    ptx::griddep_wait();
    // normalisers: one warp per beam
    for (int k = warp; k < a.beams; k += kMergeWarps) {
        const int row = row0 + k;
        if (!row_live(a, row)) continue;
        const float2* p = a.part + (size_t)row * a.splits;
        float m = -INFINITY;
        for (int s = lane; s < a.splits; s += 32) m = fmaxf(m, __ldcg(p + s).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        double sum = 0;
        for (int s = lane; s < a.splits; s += 32) {
            const float2 ms = __ldcg(p + s);
            if (ms.x != -INFINITY) sum += (double)ms.y * exp((double)ms.x - (double)m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (lane == 0) {
            s_top[k] = m == -INFINITY ? 0.f : m;
            s_shift[k] = m == -INFINITY ? 0. : (double)__ldcg(a.scores + row) - log(sum);
        }
    }
    __syncthreads();
    // Every list (a live beam's slice; a beam that ended or is at -inf) has one thread;
    // list i + kMergeThreads, ... of a thread come after its list i in the same loop.
    const int lists = a.beams * a.splits;
    constexpr int kLists = kBeamsMax * 128 / kMergeThreads;   // splits <= 128: vocab <= 2^20
    unsigned char at[kLists];                                 // how many of the list are taken
    Cand head[kLists];
    auto fetch = [&](int list, int pos) -> Cand {
        if (pos >= a.n_out) return {0ull, 0xffffffffu};
        const int k = list / a.splits, s = list - k * a.splits, row = row0 + k;
        const double score = __ldcg(a.scores + row);
        if (!row_live(a, row)) {
            if (s != 0) return {0ull, 0xffffffffu};
            if (row_ended(a, row) && score != -INFINITY) {
                // (k, eos) first, then the tokens that do not follow an end, at -inf
                if (pos == 0) return {ordered(score), (unsigned)k * a.vocab + a.eos};
                const int v = pos - 1 < a.eos ? pos - 1 : pos;
                return {ordered((double)-INFINITY), v < a.vocab ? (unsigned)k * a.vocab + v : 0xffffffffu};
            }
            return {ordered((double)-INFINITY), (unsigned)k * a.vocab + pos};
        }
        const unsigned long long key = __ldcg(a.cand + ((size_t)row * a.splits + s) * a.n_out + pos);
        if (key == 0) return {0ull, 0xffffffffu};
        const double below = (double)unordered((unsigned)(key >> 32)) - (double)s_top[k];
        return {ordered(below + s_shift[k]), (unsigned)k * a.vocab + ~(unsigned)key};
    };
#pragma unroll
    for (int i = 0; i < kLists; ++i) {
        at[i] = 0;
        head[i] = tid + i * kMergeThreads < lists ? fetch(tid + i * kMergeThreads, 0) : Cand{0ull, 0xffffffffu};
    }
    for (int o = 0; o < a.n_out; ++o) {
        Cand mine{0ull, 0xffffffffu};
#pragma unroll
        for (int i = 0; i < kLists; ++i)
            if (better(head[i], mine)) mine = head[i];
        Cand best = warp_best(mine);
        __syncthreads();
        if (lane == 0) s_best[warp] = best;
        __syncthreads();
        best = warp_best(lane < kMergeWarps ? s_best[lane] : Cand{0ull, 0xffffffffu});
        if (tid == 0) {
            const unsigned p = best.value ? best.place : 0u;
            const unsigned long long u = best.value;
            a.parents[(size_t)g * a.n_out + o] = row0 + (int)(p / (unsigned)a.vocab);
            a.tokens[(size_t)g * a.n_out + o] = (int)(p % (unsigned)a.vocab);
            a.best[(size_t)g * a.n_out + o] =
                (float)__longlong_as_double((long long)(u >> 63 ? u & 0x7fffffffffffffffull : ~u));
        }
#pragma unroll
        for (int i = 0; i < kLists; ++i)
            if (best.value != 0 && head[i].value == best.value && head[i].place == best.place)
                head[i] = fetch(tid + i * kMergeThreads, ++at[i]);
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
    if (launch_pdl(k_beam_scan, dim3(a.splits, groups * beams), dim3(kScanThreads), 0, s, a) != cudaSuccess)
        return LLAMA_ERR_CUDA;
    if (launch_pdl(k_beam_merge, dim3(groups), dim3(kMergeThreads), 0, s, a) != cudaSuccess) return LLAMA_ERR_CUDA;
    return LLAMA_OK;
}
