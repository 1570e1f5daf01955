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
// k_beam_scan streams a slice of a row through shared memory in chunks, and leaves the
// slice's maximum, its sum of exponentials and its n_out best (logit, token) pairs in order;
// k_beam_merge joins a request's slices.
//
// A slice's sum (at most kChunksMax * kChunk = 32768 terms of at most 1) is fp32: a lane's
// two sums add a chunk's 16 terms each, then the chunks; the lanes' and slices' sums are
// joined in 2^36 fixed point and everything after them is fp64, since an fp32 cumulative score
// rounds different logits to equal candidates.  In units of u = 2^-24 a term's relative error
// is 4 (ex2) and, for its distance d from the row's maximum, 2.25 d (two roundings and the
// rounded log2 e; d averages less than 14 where e^-d weighs 2^20 terms); its additions are 15 in
// the chunk, 31 over the chunks and 1 of the lane's two sums; a chunk that raises the maximum
// multiplies the sums by e^(old - new) (5, at most 31 times), as does the slices' join (6): in
// all at most 4 + 32 + 15 + 31 + 1 + 155 + 6 = 244 u, below 2^-16 in the logarithm.  (One chain
// through the slice, 512 additions, could be off by 2^-15.)
//
// Bound by the read of the logits (115 MB: 17 us at the copy rate) and by what is done to
// each of them: both launches together take 31.4 us for 32 requests of 8 beams, 128,256
// tokens and n_out = 16, and the host's call 10.7 us where there is one request.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanCtas = 3;                              // CTAs per SM
constexpr int kPerLane = 32;                              // logits per lane of a chunk
constexpr int kChunk = 32 * kPerLane;
constexpr int kScanStages = 2;                            // chunks in flight per warp
constexpr int kSplitsMax = 32;                            // slices per row
constexpr int kChunksMax = 32;                            // chunks per slice
constexpr float kFix = 68719476736.0f;                    // 2^36: sums of exponentials in fixed point
constexpr int kMergeThreads = 512;
constexpr int kMergeWarps = kMergeThreads / 32;           // and one more for the logarithms
constexpr int kMergeCap = 1024;                           // candidates ranked per request
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
    int beams, vocab, n_out, splits, rows;
    int slice_chunks;             // chunks of kChunk logits per slice
    int ahead;                    // keys of each list that the merge loads ahead
    unsigned div_out, div_splits, div_ahead;   // ceil(2^32 / n) of n_out, splits and ahead
    uint4* part;                  // [rows][splits]: slice maximum, sum of e^(z - maximum) 2^36 (64 bits)
    unsigned long long* cand;     // [rows][splits][n_out] candidate keys, decreasing
    int* parents;
    int* tokens;
    float* best;
};

// 0: a beam whose candidates its logits decide (the others are not read), 1: one that has
// ended, 2: one at -inf.  The two words are loaded together.
__device__ __forceinline__ int row_mode(const BeamArgs& a, int row) {
    const float score = __ldcg(a.scores + row);
    const int last = a.last ? __ldcg(a.last + row) : -1;   // eos >= 0 where there is a last
    return score == -INFINITY ? 2 : a.last && last == a.eos ? 1 : 0;
}

// 2^x on the special-function unit (ex2.approx.ftz: relative error 2^-22).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 lanes per instruction (sm_100 and later), each the IEEE operation.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void cp_async16(void* smem, const void* gmem, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(smem)), "l"(gmem), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(void* smem, const void* gmem, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(smem)), "l"(gmem), "r"(valid ? 4 : 0)
                 : "memory");
}
// Sum over the warp of values below 2^47 (exact: two 32-bit sums of 24-bit parts).
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
    const unsigned lo = __reduce_add_sync(kAll, (unsigned)v & 0xffffffu);
    const unsigned hi = __reduce_add_sync(kAll, (unsigned)(v >> 24));
    return ((unsigned long long)hi << 24) + lo;
}
// i / n for i * n < 2^32, with m = ceil(2^32 / n) (0 for n = 1).
__device__ __forceinline__ int fast_div(int i, unsigned m) { return m ? (int)__umulhi((unsigned)i, m) : i; }

// The lanes' keys in decreasing order (a bitonic network).
__device__ __forceinline__ unsigned exchange(unsigned key, int distance, bool larger) {
    const unsigned other = __shfl_xor_sync(kAll, key, distance);
    return larger ? max(key, other) : min(key, other);
}
__device__ __forceinline__ unsigned warp_sort(unsigned key) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int run = 2; run <= 32; run *= 2)
#pragma unroll
        for (int d = run / 2; d > 0; d /= 2) key = exchange(key, d, ((lane & d) == 0) == ((lane & run) == 0));
    return key;
}
// The n-th largest of the lanes' N keys each, n <= 32 N.
template <int N>
__device__ __forceinline__ unsigned warp_nth(const unsigned (&keys)[N], int n) {
    const unsigned first = warp_sort(keys[0]);
    if constexpr (N == 1) return __shfl_sync(kAll, first, n - 1);
    else {
        // of two decreasing runs a and b, max(a[i], b[31 - i]) are the 32 largest
        const unsigned other = __shfl_xor_sync(kAll, warp_sort(keys[1]), 31);
        const unsigned half = warp_sort(n <= 32 ? max(first, other) : min(first, other));
        return __shfl_sync(kAll, half, (n - 1) & 31);
    }
}

// Where lane holds value i of a chunk.  VEC: rows of whole 16-byte vectors, copied as
// such; a lane then holds runs of four.
template <bool VEC>
__device__ __forceinline__ int chunk_at(int lane, int i) {
    return VEC ? (i >> 2) * 128 + lane * 4 + (i & 3) : lane + i * 32;
}
// Place of value i in the lane's part of a stage (16-byte vectors, lane by lane).
__device__ __forceinline__ int stage_at(int lane, int i) { return (i >> 2) * 128 + lane * 4 + (i & 3); }

// Shared memory of a warp of the scan: the chunks in flight and the gathered candidates.
__host__ __device__ constexpr int list_cap(int n) { return n <= 32 ? 64 : 128; }   // n_out + 32 at least
__host__ __device__ constexpr int scan_warp_bytes(int n_out) { return kScanStages * kChunk * 4 + list_cap(n_out) * 8; }

// Ranks the `count` keys of a list (all different) by counting the larger ones and hands
// each key and its rank to f, a lane per key.
template <typename F>
__device__ __forceinline__ void rank_keys(const unsigned long long* list, int count, F f) {
    for (int c = threadIdx.x & 31; c < count; c += 32) {
        const unsigned long long key = list[c];
        int rank = 0;
#pragma unroll 8
        for (int i = 0; i < count; ++i) rank += list[i] > key;
        f(rank, key);
    }
}

// A warp per slice, no barrier: a row's slices are cut so that the warps of the grid take
// them in as few rounds as they can (scan_split), and a slice is walked in chunks of 1024
// logits that the lanes copy ahead, each its own values, into shared memory.
//
// The largest logits are gathered in the same walk: the n_out-th largest of the lanes'
// maxima so far bounds the n_out-th largest logit from below (taken anew when the number
// of chunks has doubled), and what reaches it is appended to a list that is ranked by
// counting at the end.  A logit costs its exponential, a maximum and a comparison, about 6
// instructions.  256 rows of 128,256 logits, 32 of them ended, n_out = 16: 25 us warm, 28 cold
// (115 MB, 4.1 TB/s; 48% of the issue slots, warps waiting on their own chains of shuffles).
// Reading the runs of the largest maxima again at the end took 4 us more (most had left
// L2), a sorted list kept per warp 33 us cold, a CTA per slice of 8192 logits with two
// barriers 34, n_out block-wide maxima 179.
//
// VEC: rows of whole 16-byte vectors.  N = 2 (n_out > 32): two maxima a lane, of the
// halves of its runs.
template <bool VEC, int N>
__global__ void __launch_bounds__(kScanThreads, kScanCtas) k_beam_scan(const BeamArgs a) {
    extern __shared__ __align__(16) uint8_t s_scan[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kCap = list_cap(32 * N);
    float* ring = reinterpret_cast<float*>(s_scan + warp * scan_warp_bytes(32 * N));
    unsigned long long* list = reinterpret_cast<unsigned long long*>(ring + kScanStages * kChunk);
    ptx::griddep_wait();
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();   // the merge waits for this grid before it reads
    const int units = a.rows * a.splits, step = gridDim.x * kScanWarps;   // below 2^21
    const unsigned lowest = ordered(-INFINITY);

    // the (unit, chunk) that is copied next; units of rows that are not read are passed over
    int pu = blockIdx.x * kScanWarps + warp, p_row = 0, p_v0 = 0, p_left = 0;
    auto enter = [&]() {   // the first chunk of unit pu, or of the next one that is read
        while (pu < units && row_mode(a, pu / a.splits) != 0) pu += step;
        if (pu < units) {
            p_row = pu / a.splits;
            p_v0 = (pu - p_row * a.splits) * a.slice_chunks * kChunk;
            p_left = a.slice_chunks;
        }
    };
    enter();
    auto prefetch = [&](int stage) {
        if (pu < units) {
            const int n = a.vocab - p_v0;
            const float* z = a.logits + (size_t)p_row * a.vocab + p_v0;
            float* to = ring + stage * kChunk;
            if (VEC && n >= kChunk) {
#pragma unroll
                for (int i = 0; i < kPerLane; i += 4) cp_async16(to + stage_at(lane, i), z + chunk_at<VEC>(lane, i), true);
            } else {
#pragma unroll
                for (int i = 0; i < kPerLane; i += VEC ? 4 : 1) {
                    const int j = chunk_at<VEC>(lane, i);
                    if constexpr (VEC) cp_async16(to + stage_at(lane, i), z + (j < n ? j : 0), j < n);
                    else cp_async4(to + stage_at(lane, i), z + (j < n ? j : 0), j < n);
                }
            }
            p_v0 += kChunk;
            if (--p_left == 0 || p_v0 >= a.vocab) {
                pu += step;
                enter();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int u = pu, at = 0;   // the unit at work, the stage of its next chunk
#pragma unroll
    for (int i = 0; i < kScanStages; ++i) prefetch(i);
    while (u < units) {
        const int row = u / a.splits, split = u - row * a.splits;
        const int begin = split * a.slice_chunks * kChunk, size = min(a.slice_chunks * kChunk, a.vocab - begin);
        const int chunks = (size + kChunk - 1) / kChunk;
        float m = -INFINITY;    // largest logit so far
        float half_max[2] = {-INFINITY, -INFINITY};   // of the lane's runs
        unsigned bound = 0;     // below no more than n_out - 1 of the slice's logits so far; 0: not known
        float bf = -INFINITY;   // as a number
        int count = 0;          // listed candidates
        unsigned long long least = 0;   // a key that n_out listed ones are not below
        uint64_t sums = 0;      // the lane's two sums of e^(x - m)
        for (int c = 0; c < chunks; ++c) {
            const int n = size - c * kChunk;
            const float* stage = ring + at * kChunk;
            asm volatile("cp.async.wait_group %0;" ::"n"(kScanStages - 1) : "memory");
            float x[kPerLane];
#pragma unroll
            for (int i = 0; i < kPerLane; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(stage + stage_at(lane, i));
                x[i] = v.x;
                x[i + 1] = v.y;
                x[i + 2] = v.z;
                x[i + 3] = v.w;
            }
            if (n < kChunk) {   // the row's last chunk
#pragma unroll
                for (int i = 0; i < kPerLane; ++i)
                    if (chunk_at<VEC>(lane, i) >= n) x[i] = -INFINITY;
            }
            float half[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float* y = x + h * (kPerLane / 2);
                half[h] = fmaxf(y[0], y[1]);
#pragma unroll
                for (int i = 2; i < kPerLane / 2; i += 2) half[h] = max3(half[h], y[i], y[i + 1]);
                half_max[h] = fmaxf(half_max[h], half[h]);
            }
            const float most = fmaxf(half[0], half[1]);
            if (__any_sync(kAll, most > m)) {
                const float now = unordered(__reduce_max_sync(kAll, ordered(most)));
                const float r = ex2((m - now) * kLog2e);   // 0 from m = -inf on
                sums = mul2(sums, pack2(r, r));
                m = now;
            }
            if (m != -INFINITY) {
                const uint64_t down = pack2(-m, -m), scale = pack2(kLog2e, kLog2e);
                uint64_t part = 0;   // of this chunk: chains of 16 terms and of 32 chunks, not one of 512
#pragma unroll
                for (int i = 0; i < kPerLane; i += 2) {
                    float y0, y1;
                    unpack2(mul2(add2(pack2(x[i], x[i + 1]), down), scale), y0, y1);
                    const uint64_t e = pack2(ex2(y0), ex2(y1));
                    part = i == 0 ? e : add2(part, e);
                }
                sums = add2(sums, part);
            }
            if ((c & (c + 1)) == 0) {   // 1, 2, 4, ... chunks
                // a lane (a half) without a logit has none in any chunk: the row ends in its first
                unsigned keys[N];
                if constexpr (N == 1) {
                    keys[0] = chunk_at<VEC>(lane, 0) < size ? ordered(fmaxf(half_max[0], half_max[1])) : 0u;
                } else {
                    keys[0] = chunk_at<VEC>(lane, 0) < size ? ordered(half_max[0]) : 0u;
                    keys[1] = chunk_at<VEC>(lane, kPerLane / 2) < size ? ordered(half_max[1]) : 0u;
                }
                const unsigned now = warp_nth<N>(keys, a.n_out);
                if (now > bound) {
                    bound = now;
                    bf = now > lowest ? unordered(now) : -INFINITY;
                }
            }
            if (__any_sync(kAll, most >= bf)) {
                unsigned hits = 0;
#pragma unroll
                for (int i = 0; i < kPerLane; ++i)
                    if (x[i] >= bf) hits |= 1u << i;
                while (__any_sync(kAll, hits != 0)) {   // every lane's next one
                    unsigned long long key = 0;
                    if (hits) {
                        const int i = __ffs(hits) - 1, j = chunk_at<VEC>(lane, i);
                        hits &= hits - 1;
                        if (j < n) key = cand_key(stage[stage_at(lane, i)], begin + c * kChunk + j);
                    }
                    const unsigned who = __ballot_sync(kAll, key > least);
                    if (key > least) list[count + __popc(who & ((1u << lane) - 1))] = key;
                    count += __popc(who);
                    __syncwarp();
                    if (count > kCap - 32) {   // keep the n_out best
                        unsigned long long mine[kCap / 32];
                        int at_rank[kCap / 32], k = 0;
#pragma unroll
                        for (int e = 0; e < kCap / 32; ++e) at_rank[e] = kCap;
                        rank_keys(list, count, [&](int rank, unsigned long long v) {
#pragma unroll
                            for (int e = 0; e < kCap / 32; ++e)
                                if (e == k) {
                                    mine[e] = v;
                                    at_rank[e] = rank;
                                }
                            ++k;
                        });
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < kCap / 32; ++e)
                            if (at_rank[e] < a.n_out) list[at_rank[e]] = mine[e];
                        __syncwarp();
                        count = min(count, a.n_out);
                        if (count == a.n_out) {
                            least = list[count - 1];
                            if ((unsigned)(least >> 32) > bound) {
                                bound = (unsigned)(least >> 32);
                                bf = bound > lowest ? unordered(bound) : -INFINITY;
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            prefetch(at);   // into the stage just read
            at = at + 1 == kScanStages ? 0 : at + 1;
        }
        const size_t slot = (size_t)row * a.splits + split;
        float sum0, sum1;
        unpack2(sums, sum0, sum1);
        // a lane's sum is at most 2^10 2^36 (32 chunks of 32 terms of at most 1)
        const unsigned long long sum = warp_sum(__float2ull_rn((sum0 + sum1) * kFix));
        if (lane == 0) a.part[slot] = make_uint4(__float_as_uint(m), 0u, (unsigned)sum, (unsigned)(sum >> 32));

        unsigned long long* out = a.cand + slot * a.n_out;
        rank_keys(list, count, [&](int rank, unsigned long long v) {
            if (rank < a.n_out) out[rank] = v;
        });
        for (int o = count + lane; o < a.n_out; o += 32) out[o] = 0;
        __syncwarp();   // the list is free again
        do u += step;
        while (u < units && row_mode(a, u / a.splits) != 0);
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
// bound comes from the lists' first keys (4096 in all; mostly that is every key), the keys
// at or above it are gathered and ranked by counting.
//
// The fp64 pipe is narrow (all keys of 8 beams, 16 slices and 16 candidates in fp64 took
// 19 us), so the bound is found in fp32 with directed roundings and a normaliser known
// within kLogSlack: a key's value rounded down, for the bound, and rounded up, against
// it -- no candidate whose fp64 value is at or above the bound is missed, and only what
// passes is computed in fp64, while a warp of its own takes the beams' logarithms in fp64
// beside the gathering.  The keys are loaded ahead of all that.
constexpr int kMergeKeys = 8;                    // keys per lane loaded ahead
// Above the error of score - logf(total): logf is off by at most 2 units in the last
// place of a value below 32 (2^-18), the rest by 2^-22 of the result.
constexpr float kLogSlack = 1.0f / 131072.0f;    // 2^-17

__global__ void __launch_bounds__(kMergeThreads + 32) k_beam_merge(const BeamArgs a) {
    // a live beam's largest logit, and its score - log sum e^(z - largest): kept apart, since
    // next to a mask of the type's lowest value a score would be lost
    __shared__ float s_top[kBeamsMax], s_score[kBeamsMax];
    __shared__ double s_shift[kBeamsMax];
    __shared__ unsigned long long s_total[kBeamsMax];
    __shared__ int s_mode[kBeamsMax];       // 0: live, 1: ended, 2: at -inf
    __shared__ float s_up[kBeamsMax], s_down[kBeamsMax];   // bounds of s_shift
    __shared__ unsigned s_first[4][kMergeWarps];
    __shared__ unsigned long long s_key[kMergeCap], s_value[kMergeCap];
    __shared__ unsigned s_place[kMergeCap];
    __shared__ Cand s_best[kMergeWarps + 1];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.x;
    const int row0 = g * a.beams;
    const int lists = a.beams * a.splits, total = lists * a.n_out;
    const unsigned lowest = ordered(-INFINITY);
    const unsigned long long* cand = a.cand + (size_t)row0 * a.splits * a.n_out;
    ptx::griddep_wait();
    if (tid == 0) s_n = 0;
    // what a row that is not read left in its place is not looked at
    // Warp w takes lists w, w + 16, ...: a beam's slices go to different warps.
    unsigned long long ahead[kMergeKeys];
    auto place = [&](int i, int& list, int& pos) {   // of a lane's i-th key
        const int r = i * 32 + lane, j = fast_div(r, a.div_ahead);
        list = warp + kMergeWarps * j;
        pos = r - j * a.ahead;
        return warp < kMergeWarps && list < lists;
    };
#pragma unroll
    for (int i = 0; i < kMergeKeys; ++i) {
        int list, pos;
        ahead[i] = place(i, list, pos) ? __ldcg(cand + (size_t)list * a.n_out + pos) : 0ull;
    }
    // normalisers: the slices' sums, one warp per beam
    for (int k = warp; k < a.beams; k += kMergeWarps + 1) {
        const int row = row0 + k;
        const uint4* p = a.part + (size_t)row * a.splits;
        static_assert(kSplitsMax == 32, "a slice per lane");
        const uint4 ms = lane < a.splits ? __ldcg(p + lane) : make_uint4(0xff800000u, 0u, 0u, 0u);
        const int mode = row_mode(a, row);
        const float score = __ldcg(a.scores + row);
        const float m = unordered(__reduce_max_sync(kAll, ordered(__uint_as_float(ms.x))));
        if (mode != 0 || m == -INFINITY) {   // no logit decides: at the score, or at -inf
            if (lane == 0) {
                s_mode[k] = mode;
                s_top[k] = 0.f;
                s_total[k] = 0;
                s_score[k] = s_up[k] = s_down[k] = score;
            }
            continue;
        }
        const float t = (float)(((unsigned long long)ms.w << 32) | ms.z);   // at most 2^51
        unsigned long long sum = __float2ull_rn(t * ex2((__uint_as_float(ms.x) - m) * kLog2e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (lane == 0) {
            const float near = score - logf((float)sum * (1.f / kFix));
            const float slack = fmaf(fabsf(near), 1.0f / 4194304.0f, kLogSlack);
            s_mode[k] = 0;
            s_top[k] = m;
            s_total[k] = sum;
            s_score[k] = score;
            s_up[k] = __fadd_ru(near, slack);
            s_down[k] = __fsub_rd(near, slack);
        }
    }
    __syncthreads();
    // the value of list's candidate `pos`, its key given, rounded up or down
    auto value32 = [&](int list, int pos, unsigned long long key, bool up) -> unsigned {
        const int k = fast_div(list, a.div_splits);
        if (s_mode[k] != 0) {
            if (list != k * a.splits) return 0u;
            return ordered(s_mode[k] == 1 && pos == 0 ? s_score[k] : -INFINITY);
        }
        if (key == 0) return 0u;
        const float z = unordered((unsigned)(key >> 32));
        return ordered(up ? __fadd_ru(__fsub_ru(z, s_top[k]), s_up[k]) : __fadd_rd(__fsub_rd(z, s_top[k]), s_down[k]));
    };
    // the candidate itself (s_shift written)
    auto candidate = [&](int list, int pos, unsigned long long key) -> Cand {
        const int k = fast_div(list, a.div_splits);
        const unsigned base = (unsigned)k * a.vocab;
        if (s_mode[k] == 1) {
            // (k, eos) first, then the tokens that do not follow an end, at -inf
            if (pos == 0) return {ordered((double)s_score[k]), base + a.eos};
            return {ordered((double)-INFINITY), base + (pos - 1 < a.eos ? pos - 1 : pos)};
        }
        if (s_mode[k] == 2) return {ordered((double)-INFINITY), base + pos};
        const double below = (double)unordered((unsigned)(key >> 32)) - (double)s_top[k];
        return {ordered(below + s_shift[k]), base + ~(unsigned)key};
    };
    if (warp == kMergeWarps) {   // a lane per beam: one warp's fp64 instructions serve all
        if (lane < a.beams)
            s_shift[lane] = s_total[lane] == 0 ? (double)s_score[lane]
                                               : (double)s_score[lane] - log((double)s_total[lane] * (1. / kFix));
    } else {
        // The bound: of the lanes' best values, rounded down, every warp's first two (four for
        // n_out > 32), and of those the n_out-th.
        unsigned mine = 0;
#pragma unroll
        for (int i = 0; i < kMergeKeys; ++i) {
            int list, pos;
            if (place(i, list, pos)) mine = max(mine, value32(list, pos, ahead[i], false));
        }
        mine = warp_sort(mine);
        if (lane < 4) s_first[lane][warp] = mine;
        ptx::named_bar_sync(1, kMergeThreads);
        static_assert(kMergeWarps == 16 && kOutMax == 64, "two lanes per warp's first keys");
        const unsigned pair[2] = {s_first[lane >> 4][lane & 15], s_first[2 + (lane >> 4)][lane & 15]};
        const unsigned one[1] = {pair[0]};
        unsigned bound = a.n_out <= 32 ? warp_nth<1>(one, a.n_out) : warp_nth<2>(pair, a.n_out);
        // Candidates at -inf count only where the others are fewer than n_out (a first step's
        // idle beams hold most of the lists' heads at -inf or empty, and so the bound down).
        bound = max(bound, lowest + 1);
        while (true) {
            auto gather = [&](int list, int pos, unsigned long long key) {
                if (value32(list, pos, key, true) >= bound) {
                    const int p = atomicAdd(&s_n, 1);
                    if (p < kMergeCap) {
                        s_place[p] = list * a.n_out + pos;
                        s_key[p] = key;
                    }
                }
            };
#pragma unroll
            for (int i = 0; i < kMergeKeys; ++i) {
                int list, pos;
                if (place(i, list, pos)) gather(list, pos, ahead[i]);
            }
            const int rest = a.n_out - a.ahead;   // of each list, not loaded yet
            for (int i = tid; i < lists * rest; i += kMergeThreads) {
                const int list = i / rest, pos = a.ahead + i - list * rest;
                gather(list, pos, __ldcg(cand + (size_t)list * a.n_out + pos));
            }
            ptx::named_bar_sync(1, kMergeThreads);
            if (s_n >= a.n_out || bound == lowest) break;
            ptx::named_bar_sync(1, kMergeThreads);   // everyone has read the count
            if (tid == 0) s_n = 0;
            ptx::named_bar_sync(1, kMergeThreads);
            bound = lowest;
        }
    }
    __syncthreads();
    const int found = s_n;
    auto emit = [&](int o, const Cand& c) {
        const size_t at = (size_t)g * a.n_out + o;
        a.parents[at] = row0 + (int)(c.place / (unsigned)a.vocab);
        a.tokens[at] = (int)(c.place % (unsigned)a.vocab);
        a.best[at] = (float)__longlong_as_double(
            (long long)(c.value >> 63 ? c.value & 0x7fffffffffffffffull : ~c.value));
    };
    if (found <= kMergeCap) {
        for (int c = tid; c < found; c += kMergeThreads + 32) {
            const int i = s_place[c], list = fast_div(i, a.div_out);
            const Cand x = candidate(list, i - list * a.n_out, s_key[c]);
            s_value[c] = x.value;
            s_place[c] = x.place;
        }
        __syncthreads();
        for (int c = warp; c < found; c += kMergeWarps + 1) {
            const Cand x{s_value[c], s_place[c]};
            int rank = 0;
            for (int i = 0; i < found; i += 32) {
                const int j = min(i + lane, found - 1);
                rank += __popc(__ballot_sync(kAll, i + lane < found && better(Cand{s_value[j], s_place[j]}, x)));
            }
            if (lane == 0 && rank < a.n_out) emit(rank, x);
        }
        // only logits that are no numbers leave places open: they get the group's first beam at -inf
        for (int o = found + tid; o < a.n_out; o += kMergeThreads + 32) emit(o, Cand{ordered((double)-INFINITY), 0u});
        return;
    }
    // many equal candidates: n_out rounds over all that come after the last one taken
    Cand last{~0ull, 0u};
    for (int o = 0; o < a.n_out; ++o) {
        Cand best{0ull, 0xffffffffu};
        for (int i = tid; i < total; i += kMergeThreads + 32) {
            const int list = fast_div(i, a.div_out), pos = i - list * a.n_out;
            const unsigned long long key = __ldcg(cand + i);
            if (value32(list, pos, key, true) < lowest) continue;   // none
            const Cand c = candidate(list, pos, key);
            if (better(last, c) && better(c, best)) best = c;
        }
        best = warp_best(best);
        __syncthreads();
        if (lane == 0) s_best[warp] = best;
        __syncthreads();
        last = warp_best(lane <= kMergeWarps ? s_best[lane] : Cand{0ull, 0xffffffffu});
        if (tid == 0) emit(o, last);
    }
}

// Slices per row, and chunks per slice: the rows' slices are taken by the grid's warps in
// rounds, a round lasting as long as a slice; each slice costs about two chunks more than
// its own (its first list), and more slices make the merge longer.  On equal time, fewer.
struct Split { int splits, chunks; };
Split scan_split(int rows, int vocab, int warps) {
    const int total = (vocab + kChunk - 1) / kChunk;
    Split best{0, 0};
    long long cost = 0;
    for (int s = 1; s <= kSplitsMax && s <= total; ++s) {
        const int chunks = (total + s - 1) / s;
        if (chunks > kChunksMax) continue;
        if ((total + chunks - 1) / chunks != s) continue;   // the same chunks with fewer slices
        const long long rounds = ((long long)rows * s + warps - 1) / warps, c = rounds * (chunks + 2);
        if (best.splits == 0 || c < cost) {
            best = {s, chunks};
            cost = c;
        }
    }
    return best;
}
int slices_at_most(int vocab) { return std::min((vocab + kChunk - 1) / kChunk, kSplitsMax); }
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
    const size_t lists = (size_t)groups * beams * slices_at_most(vocab);
    return align256(lists * sizeof(uint4)) + align256(lists * n_out * sizeof(unsigned long long));
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
    const int max_warps = device_sm_count() * kScanCtas * kScanWarps;
    const Split cut = scan_split(groups * beams, vocab, max_warps);
    a.splits = cut.splits;
    a.slice_chunks = cut.chunks;
    a.part = (uint4*)ws;
    a.cand = (unsigned long long*)((uint8_t*)ws + align256((size_t)groups * beams * a.splits * sizeof(uint4)));
    a.parents = parents;
    a.tokens = tokens;
    a.best = out_scores;
    cudaStream_t s = (cudaStream_t)stream;
    a.rows = groups * beams;
    a.div_out = n_out > 1 ? (unsigned)(((1ull << 32) + n_out - 1) / n_out) : 0u;
    a.ahead = std::min(n_out, kMergeKeys * 32 / ((beams * a.splits + kMergeWarps - 1) / kMergeWarps));
    a.div_ahead = a.ahead > 1 ? (unsigned)(((1ull << 32) + a.ahead - 1) / a.ahead) : 0u;
    a.div_splits = a.splits > 1 ? (unsigned)(((1ull << 32) + a.splits - 1) / a.splits) : 0u;
    const bool vec = vocab % 4 == 0 && ((uintptr_t)logits & 15) == 0;
    const auto scan = n_out <= 32 ? (vec ? k_beam_scan<true, 1> : k_beam_scan<false, 1>)
                                  : (vec ? k_beam_scan<true, 2> : k_beam_scan<false, 2>);
    cudaError_t e = kernel_setup_once((const void*)scan, [](const void* kern) {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kScanWarps * scan_warp_bytes(kOutMax));
    });
    if (e != cudaSuccess) return LLAMA_ERR_CUDA;
    const int units = a.rows * a.splits;
    const unsigned ctas = (unsigned)std::min((units + kScanWarps - 1) / kScanWarps, device_sm_count() * kScanCtas);
    if (launch_pdl(scan, dim3(ctas), dim3(kScanThreads), (size_t)kScanWarps * scan_warp_bytes(n_out), s, a) !=
        cudaSuccess)
        return LLAMA_ERR_CUDA;
    if (launch_pdl(k_beam_merge, dim3(groups), dim3(kMergeThreads + 32), 0, s, a) != cudaSuccess) return LLAMA_ERR_CUDA;
    return LLAMA_OK;
}
