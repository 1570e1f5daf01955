// The work of a chunk attention call, shared by its kernels: which keys of which query tile a CTA takes.
//
// A tile is `tq` consecutive new tokens of a sequence under one KV head (tq x the group's heads rows);
// its work is the keys that its last token attends and a constant for starting and storing a tile.  Lengths
// and counts are read on the device, so both ways of dealing tiles out hold for any mixture of sequences
// under any bound:
//   - many tiles: whole tiles in rounds, the longest of a sequence first (few rounds: of all sequences) and every other
//     round from the other end.  CTAs then walk the keys of a head at about the same time, and find them in L2
//     (stretches of a line as below: 8192 tokens of 32 / 8 heads 920 us, in rounds 755, one tile a CTA at a time);
//   - few: all tiles -- sequences in order, their KV heads, their tiles -- lie one after another on a line of length
//     W, and CTA i of n takes the stretch from i W / n on, cut at chunks of kAttnChunk keys (chunk_cut): a
//     tile that crosses the end of a stretch is shared by several CTAs, each of which leaves the softmax
//     partial (m, l, o) of its chunks, and a second kernel joins them.
#pragma once
#include <algorithm>

#include "common.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace llama {

// Sequences and CTAs of a launch, and the query rows of a tile
constexpr int kTcSeqs = 1024, kTcCtas = 152, kTcRows = 256;
constexpr int kF32Seqs = 256, kF32Ctas = 304, kF32Rows = 64, kF32Keys = 64;
constexpr int kChunkMaxCtas = std::max(kTcCtas, kF32Ctas);

// A sum that goes on over millions of keys loses a little with each: O in tensor memory, whose additions are cut off, came out
// 0.6 % small over 2^20 positions and 10 % over 2^24; products added up one by one in fp32 were off by up to 1 % over 2^20.
// So a row's O and l are carried over to second sums, O in fp32 in the workspace, every kTcCarry chunks of a piece (2^-11 at
// most lost in each) and every kF32Carry blocks of kF32Keys keys.
constexpr int kTcCarry = 512, kF32Carry = 32;

// How a type's tiles are dealt out.
struct ChunkDeal {
    int seqs, ctas, rows;
    int carry_keys;      // a row's sums over so many keys are carried over (see ChunkArgs::carry)
    int tq;              // tokens per tile
    int join_keys;       // work (keys) per CTA that the partials and their joining cost
    int min_stretch;     // the least work of a CTA (keys) for which tiles are split
    float pieces;        // ... and the pieces of a tile of c chunks, at most: pieces * sqrt(c)
};
inline ChunkDeal chunk_deal_tc(int n_rep) { return {kTcSeqs, kTcCtas, kTcRows, kTcCarry * kAttnChunk, 2 * (kTcRows / 2 / n_rep), 768, 512, 2.f}; }
// two CTAs an SM where shared memory has room for them (244 tokens behind 34056, 4 / 2 heads of 64: 318 us with one, 276)
constexpr int f32_ctas_per_sm(int head_dim) { return head_dim <= 64 ? 2 : 1; }
inline ChunkDeal chunk_deal_f32(int n_rep, int head_dim) {
    return {kF32Seqs, kF32Ctas / 2 * f32_ctas_per_sm(head_dim), kF32Rows, kF32Carry * kF32Keys, kF32Rows / n_rep, 64, 256, 4.f};
}

struct ChunkArgs {
    const void* q;       // [batch, tokens, n_heads, head_dim]
    void* o;
    const void* kc;
    const void* vc;
    int batch, tokens, n_heads, n_kv_heads, max_pos;
    const int* start;
    const int* count;
    PageTable pages;
    float scale_log2;
    int tq, join_keys, min_stretch;   // see ChunkDeal
    float pieces;
    int split_ctas;      // CTAs that stretches go to, at most: the workspace has partials of so many
    float* partial;      // [2 CTAs][halves of a tile][head_dim / 4][rows of a half] float4
    float2* part_ml;     // [2 CTAs][halves][rows]
    float* carry;        // [CTAs][halves][head_dim / 4][rows of a half] float4: O as carried over
    int4* cuts;          // [CTAs]: the tile that a CTA's stretch begins in {b, g, tile} and its first chunk of it ...
    int* cut_tokens;     // ... and the tile's tokens
    int* err;
};
cudaError_t launch_chunk_tc(const ChunkArgs& a, int head_dim, cudaStream_t s);    // bf16
cudaError_t launch_chunk_f32(const ChunkArgs& a, int head_dim, cudaStream_t s);

// Work of a tile in keys, beside the keys themselves: filling and draining the pipeline, q and o.
constexpr int kTileKeys = 128;
// The least chunks of a piece: what joining costs.
constexpr int kMinPiece = 2;
// Tiles of fewer positions have fewer chunks than two pieces and are never split (the join costs 3 us without any).
constexpr int kNeverSplit = (2 * kMinPiece - 1) * kAttnChunk + 1;
// Tiles per CTA from which on they are dealt out whole ...
constexpr int kRounds = 4;
// ... and fewer are too where the last round's idle CTAs cost less than join_keys per CTA (2048 tokens of 32 / 8 heads,
// 256 tiles: split 65 us, whole 40).  Those of several sequences go in the order of all tiles' lengths (8 sequences of
// mixed starts and counts, 32 / 8 heads, some 300 tiles: sequence by sequence 79 us, so 63), where more tiles than CTAs make an
// order matter.  A warp finds a tile by bisection over the lengths (32 sequences of 4 tokens, nothing to gain: 0.3 us in
// 39); a lane holds kSortSeqs / 32 sequences.
constexpr int kSortSeqs = 64;

// The sequences of a launch, N at most (shared memory).
template <int N>
struct ChunkSeqs {
    static constexpr int kMost = N;
    long long pre[N + 1];   // work of the sequences before, one KV head
    int start[N], count[N];
    int tiles[N + 1];       // tiles of the sequences before, one KV head
};

// Work of the first n tiles (all of tq tokens) of a sequence.
__device__ __forceinline__ long long tiles_work(int start, int tq, int n) {
    return (long long)n * (start + kTileKeys) + (long long)tq * n * (n + 1) / 2;
}

// Fills s (one warp).  A sequence whose words are out of range has no tile; `record`: it is recorded.
template <class Seqs>
__device__ __forceinline__ void chunk_seqs(const ChunkArgs& a, Seqs& s, bool record) {
    const int lane = threadIdx.x & 31;
    long long run = 0;
    int run_tiles = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        int start = 0, count = 0;
        if (b < a.batch) {
            start = __ldcg(a.start + b);
            count = __ldcg(a.count + b);
            if (start < 0 || count < 0 || count > a.tokens || (long long)start + count > a.max_pos) {
                if (record) record_error(a.err, LLAMA_ERR_POS_RANGE);
                count = 0;
            }
            s.start[b] = start;
            s.count[b] = count;
        }
        const int n = (count + a.tq - 1) / a.tq;
        long long w = n > 0 ? tiles_work(start, a.tq, n - 1) + start + count + kTileKeys : 0;
        int t = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, w, o);
            const int u = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) {
                w += v;
                t += u;
            }
        }
        if (b < a.batch) {
            s.pre[b + 1] = run + w;
            s.tiles[b + 1] = run_tiles + t;
        }
        run += __shfl_sync(0xffffffffu, w, 31);
        run_tiles += __shfl_sync(0xffffffffu, t, 31);
    }
    if (lane == 0) {
        s.pre[0] = 0;
        s.tiles[0] = 0;
    }
}

// The chunk of a tile (n chunks, `work` in all) at which a stretch ends that ends `x` behind the tile's
// beginning: 0 and n when the tile belongs to one side whole.
__device__ __forceinline__ int chunk_cut(long long x, int n, long long work) {
    if (x <= 0) return 0;
    if (x >= work) return n;
    const int c = (int)((x + kAttnChunk / 2) / kAttnChunk);
    return c < kMinPiece ? 0 : c > n - kMinPiece ? n : c;
}

// Chunks [c0, c1) of one tile.
struct ChunkPiece {
    int b, g, y;
    int t0, t1;       // tokens
    int pos0;         // position of t0
    int kv_last;      // position of t1 - 1
    int c0, c1, n;    // of n chunks
    int from, to;     // the piece that they are a part of (k_attn_chunk)
};

// The last x of 0 .. n - 1 for which pred holds; it holds for 0, and for none behind one that it does not hold for.
// The whole warp, 32 probes at a time (a bisection takes the latency of each of its probes).
template <class Pred>
__device__ __forceinline__ int last_that(int n, Pred pred) {
    int lo = 0;
    while (n > 1) {
        const int by = (n + 31) >> 5, x = (threadIdx.x & 31) * by;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, x < n && pred(lo + x)));
        lo += k * by;
        n = min(by, n - k * by);
    }
    return lo;
}

// A CTA's pieces in order.  The whole warp walks: the CTA waits for the first piece, and one lane's 64-bit divisions
// and bisections took 2.5 us of it.
template <class Seqs>
struct ChunkWalk {
    const Seqs& s;
    int batch, n_kv, tq, cta, n_ctas;
    bool rounds, sorted;
    int j;                 // rounds: the next one
    // sorted: the least and most keys of a tile, and the sequences of the lane
    int shortest, longest;
    unsigned tq_inverse;
    int lane_start[kSortSeqs / 32], lane_count[kSortSeqs / 32], lane_tiles[kSortSeqs / 32];
    long long w, w0, w1;   // beginning of the tile at hand, the stretch
    int b, g, y, n_qt, start, count;

    __device__ __forceinline__ ChunkWalk(const ChunkArgs& a, const Seqs& seqs, int cta_, int n_ctas_)
        : s(seqs), batch(a.batch), n_kv(a.n_kv_heads), tq(a.tq), cta(cta_), n_ctas(n_ctas_) {
        const long long total = s.pre[batch] * n_kv;
        b = batch;
        j = 0;
        w = w0 = w1 = 0;
        g = y = n_qt = start = count = 0;
        const int tiles = s.tiles[batch] * n_kv;
        // work of a CTA, if all have the same and if it takes the tiles of a CTA in rounds
        const int n_rounds = 1 + (tiles > n_ctas) + (tiles > 2 * n_ctas) + (tiles > 3 * n_ctas);
        const float each_f = __fdividef((float)total, (float)n_ctas);
        sorted = false;
        rounds = tiles >= kRounds * n_ctas;
        if (!rounds && tiles > 0 && (float)n_rounds * (float)total <= (each_f + a.join_keys) * (float)tiles) {
            rounds = true;
            sorted = tiles > n_ctas && batch > 1 && batch <= kSortSeqs;
        }
        if (sorted) {
            tq_inverse = 0x80000000u / (unsigned)tq + 1;
            longest = 0;
            shortest = 0x7fffffff;
#pragma unroll
            for (int i = 0; i < kSortSeqs / 32; ++i) {
                const int x = 32 * i + (threadIdx.x & 31), n = x < batch ? s.count[x] : 0;
                lane_count[i] = n > 0 ? n : -1;
                lane_start[i] = n > 0 ? s.start[x] : 0x3fffffff;
                lane_tiles[i] = n > 0 ? s.tiles[x + 1] - s.tiles[x] : 0;
                if (n > 0) {
                    longest = max(longest, lane_start[i] + n);
                    shortest = min(shortest, lane_start[i] + min(tq, n));
                }
            }
            longest = __reduce_max_sync(0xffffffffu, longest);
            shortest = __reduce_min_sync(0xffffffffu, shortest);
        }
        if (rounds) return;
        // The join takes a tile's pieces a batch at a time, a round trip each: p pieces of c / p chunks and their joining take
        // the least time at a p that grows with the root of c (4 tokens of one KV head behind 32768, bf16: split over all CTAs
        // 31 us, so 25; behind 131072 58 and 43; fp32 58 and 50)
        const float work = __fdividef((float)total, (float)a.min_stretch);
        float most;   // (with sqrtf, whose code is longer, the bf16 kernel's 8192 tokens took 374 us, so 356)
        asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(most) : "f"((float)total * (float)tiles * (1.f / kAttnChunk)));
        most *= a.pieces;
        const int n = min(min(n_ctas, a.split_ctas), max(tiles, (int)fminf(work, most)));
        if (cta >= n || total == 0) return;
        // every CTA has the same `each`, whatever its last bits
        const long long each = (long long)__fdividef((float)total, (float)n);
        w0 = each * cta;
        w1 = cta == n - 1 ? total : w0 + each;
        // the last sequence that begins at or before w0: one with work
        b = last_that(batch, [&](int x) { return s.pre[x] * n_kv <= w0; });
        load();
        const long long one = s.pre[b + 1] - s.pre[b];
        long long r = w0 - s.pre[b] * n_kv;
        g = last_that(n_kv, [&](int x) { return one * x <= r; });
        r -= g * one;
        y = last_that(n_qt, [&](int x) { return tiles_work(start, tq, x) <= r; });
        w = w0 - r + tiles_work(start, tq, y);
    }
    __device__ __forceinline__ void load() {
        start = s.start[b];
        count = s.count[b];
        n_qt = s.tiles[b + 1] - s.tiles[b];
    }
    __device__ __forceinline__ void tile(ChunkPiece& p) const {
        p.b = b;
        p.g = g;
        p.y = y;
        p.t0 = y * tq;
        p.t1 = min(p.t0 + tq, count);
        p.pos0 = start + p.t0;
        p.kv_last = start + p.t1 - 1;
        p.n = p.kv_last / kAttnChunk + 1;
        p.c0 = 0;
        p.c1 = p.n;
    }
    // Tiles of one of the lane's sequences under one KV head with `keys` keys or more (a tile has
    // start + min((y + 1) tq, count)).  A division by tq is a product: below 2^23 x / tq = x (2^31 / tq + 1) / 2^31, and
    // the tiles of a sorted launch hold fewer tokens.
    __device__ __forceinline__ int tiles_from(int i, int keys) const {
        const int over = keys - lane_start[i];
        const int n = lane_tiles[i] - (int)__umulhi(2u * (unsigned)max(over - 1, 0), tq_inverse);
        return over > lane_count[i] ? 0 : n;
    }
    __device__ __forceinline__ int all_from(int keys) const {
        int n = 0;
#pragma unroll
        for (int i = 0; i < kSortSeqs / 32; ++i) n += tiles_from(i, keys);
        return __reduce_add_sync(0xffffffffu, n) * n_kv;
    }
    // Tile number l of the tiles in order of decreasing keys (equal ones: by sequence, then KV head).
    __device__ __forceinline__ void pick_sorted(int l) {
        int lo = shortest, hi = longest, above = 0;   // the most keys that more than l tiles have; tiles of more
        while (lo < hi) {
            const int mid = lo + ((hi - lo + 1) >> 1), n = all_from(mid);
            if (n > l) {
                lo = mid;
            } else {
                hi = mid - 1;
                above = n;
            }
        }
        const int r = l - above;   // among the tiles of `lo` keys, one per sequence and head at most
        g = r % n_kv;
        int left = r / n_kv, to_end = 0;
#pragma unroll
        for (int i = 0; i < kSortSeqs / 32; ++i) {
            const int n = tiles_from(i, lo);
            const unsigned word = __ballot_sync(0xffffffffu, n > tiles_from(i, lo + 1));
            if (left >= 0 && left < __popc(word)) {
                const int of = __fns(word, 0, left + 1);
                b = 32 * i + of;
                to_end = __shfl_sync(0xffffffffu, n, of);
            }
            left = left < __popc(word) ? -1 : left - __popc(word);
        }
        load();
        y = n_qt - to_end;
    }
    // The next piece; false behind the last.
    __device__ __forceinline__ bool next(ChunkPiece& p) {
        if (sorted) {
            const int l = j * n_ctas + (j & 1 ? n_ctas - 1 - cta : cta);
            ++j;
            if (l >= s.tiles[batch] * n_kv) return false;
            pick_sorted(l);
            tile(p);
            return true;
        }
        if (rounds) {
            const int l = j * n_ctas + (j & 1 ? n_ctas - 1 - cta : cta);
            ++j;
            if (l >= s.tiles[batch] * n_kv) return false;
            b = last_that(batch, [&](int x) { return s.tiles[x] * n_kv <= l; });
            load();
            const int r = l - s.tiles[b] * n_kv;
            g = r % n_kv;
            y = n_qt - 1 - r / n_kv;
            tile(p);
            return true;
        }
        while (b < batch && w < w1) {
            tile(p);
            const long long work = p.kv_last + 1 + kTileKeys;
            p.c0 = chunk_cut(w0 - w, p.n, work);
            p.c1 = chunk_cut(w1 - w, p.n, work);
            w += work;
            if (++y == n_qt) {
                y = 0;
                if (++g == n_kv) {
                    g = 0;
                    do ++b;
                    while (b < batch && s.count[b] == 0);
                    if (b < batch) load();
                }
            }
            if (p.c0 < p.c1) return true;
        }
        return false;
    }
    // Where the stretch begins (chunk 0 when it begins with a tile).  Before the first next().
    __device__ __forceinline__ void begin(const ChunkArgs& a) const {
        int4 cut = make_int4(0, 0, 0, 0);
        int tokens = 0;
        if (b < batch) {
            tokens = min(tq, count - y * tq);
            const int kv_last = start + y * tq + tokens - 1, n = kv_last / kAttnChunk + 1;
            const int c = chunk_cut(w0 - w, n, (long long)kv_last + 1 + kTileKeys);
            cut = make_int4(b, g, y, c < n ? c : 0);
        }
        if (threadIdx.x % 32 == 0) {
            a.cuts[cta] = cut;
            a.cut_tokens[cta] = tokens;
        }
    }
};

namespace {

// Joins the pieces of the split tiles, in ascending order: o = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p, M the
// largest m_p.  Every CTA reads all cuts and counts the split tiles; an item is one half of a tile and kJoinCols columns,
// thread = row (rows of 64: two column groups).  The loads of several pieces go out together.  Bound by the partials (100
// tokens behind 8192, 32 / 8 heads: 20 MB, written and read within L2) and the latency of two loads before them.
constexpr int kJoinCols = 8, kJoinBatch = 6;
constexpr int kJoinThreads = 128;

__device__ __forceinline__ void store_joined(bf16* dst, const float (&o)[kJoinCols], float inv) {
    uint32_t packed[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 v2 = __floats2bfloat162_rn(o[2 * q] * inv, o[2 * q + 1] * inv);
        packed[q] = *reinterpret_cast<const uint32_t*>(&v2);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
}
__device__ __forceinline__ void store_joined(float* dst, const float (&o)[kJoinCols], float inv) {
#pragma unroll
    for (int q = 0; q < kJoinCols; q += 4)
        *reinterpret_cast<float4*>(dst + q) = make_float4(o[q] * inv, o[q + 1] * inv, o[q + 2] * inv, o[q + 3] * inv);
}

// HALVES of ROWS rows each.
template <typename T, int DH, int HALVES, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) k_attn_chunk_join(const ChunkArgs a, int n_ctas) {
    __shared__ int4 s_cut[kChunkMaxCtas];
    __shared__ int s_tokens[kChunkMaxCtas];
    constexpr int kEach = (kChunkMaxCtas + kJoinThreads - 1) / kJoinThreads, kWords = kEach * (kJoinThreads / 32);
    __shared__ unsigned s_word[kWords];   // bit i: the first CTA that begins inside its tile is CTA i
    auto same_tile = [](const int4& c, const int4& d) { return c.x == d.x && c.y == d.y && c.z == d.z; };
    ptx::griddep_wait();
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
        const int i = x * kJoinThreads + threadIdx.x;
        bool first = false;
        if (i < n_ctas) {
            const int4 cut = __ldcg(a.cuts + i), before = __ldcg(a.cuts + max(i - 1, 0));
            s_cut[i] = cut;
            s_tokens[i] = __ldcg(a.cut_tokens + i);
            first = cut.w > 0 && !(before.w > 0 && same_tile(cut, before));   // CTA 0 begins with a tile
        }
        const unsigned word = __ballot_sync(0xffffffffu, first);
        if ((threadIdx.x & 31) == 0) s_word[i >> 5] = word;
    }
    __syncthreads();
    int n_split = 0;
#pragma unroll
    for (int w = 0; w < kWords; ++w) n_split += __popc(s_word[w]);
    // CTA j begins inside the tile that CTA i begins inside of
    auto same = [&](int i, int j) { return s_cut[j].w > 0 && same_tile(s_cut[i], s_cut[j]); };
    constexpr int kCols = DH / kJoinCols, kSets = kJoinThreads / ROWS;   // column groups; of an item
    const int n_rep = a.n_heads / a.n_kv_heads, tqh = a.tq / HALVES, row = threadIdx.x % ROWS, t_local = row / n_rep;
    const int items = n_split * HALVES * (kCols / kSets);
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int cols = item % (kCols / kSets) * kSets + threadIdx.x / ROWS, x = item / (kCols / kSets), half = x % HALVES;
        int i = x / HALVES, w = 0;   // the CTA of the i-th bit
        for (; i >= __popc(s_word[w]); ++w) i -= __popc(s_word[w]);
        i = w * 32 + __fns(s_word[w], 0, i + 1);
        const int4 cut = s_cut[i];
        const int t = cut.z * a.tq + half * tqh + t_local;
        if (t_local >= tqh || half * tqh + t_local >= s_tokens[i]) continue;
        int end = i + 1;   // CTAs that begin in the tile: i .. end - 1
        while (end < n_ctas && same(i, end)) ++end;
        // piece k of end - i + 1: CTA i - 1's last, then the first ones of CTAs i, i + 1, ...; a piece is empty where the
        // next begins at the same chunk
        auto slot_of = [&](int k) { return k == 0 ? 2 * (i - 1) + 1 : 2 * (i + k - 1); };
        auto is_empty = [&](int k) {
            const int j = i + k - 1;
            return k > 0 && j + 1 < end && s_cut[j + 1].w == s_cut[j].w;
        };
        const int n = end - i + 1;
        float M = -INFINITY, L = 0.f;
        float o[kJoinCols];
#pragma unroll
        for (int e = 0; e < kJoinCols; ++e) o[e] = 0.f;
        for (int k0 = 0; k0 < n; k0 += kJoinBatch) {
            float2 ml[kJoinBatch];
            float4 v[kJoinBatch][kJoinCols / 4];
#pragma unroll
            for (int x = 0; x < kJoinBatch; ++x) {
                if (k0 + x >= n) break;
                ml[x] = __ldcg(a.part_ml + (HALVES * slot_of(k0 + x) + half) * ROWS + row);
                const float4* part =
                    reinterpret_cast<const float4*>(a.partial + (size_t)(HALVES * slot_of(k0 + x) + half) * (ROWS * DH)) + row;
#pragma unroll
                for (int q = 0; q < kJoinCols / 4; ++q) v[x][q] = __ldcg(part + (cols * (kJoinCols / 4) + q) * ROWS);
            }
#pragma unroll
            for (int x = 0; x < kJoinBatch; ++x) {
                if (k0 + x >= n) break;
                if (is_empty(k0 + x)) continue;   // its part is not written
                // a piece without a key above -inf has no weight; 0 times an infinity or a NaN among its values is NaN
                const float Mn = fmaxf(M, ml[x].x);
                const float c = M == -INFINITY ? 0.f : exp2f(M - Mn), w = ml[x].x == -INFINITY ? 0.f : exp2f(ml[x].x - Mn);
                M = Mn;
                L = fmaf(L, c, ml[x].y * w);
#pragma unroll
                for (int q = 0; q < kJoinCols / 4; ++q) {
                    o[4 * q] = fmaf(o[4 * q], c, v[x][q].x * w);
                    o[4 * q + 1] = fmaf(o[4 * q + 1], c, v[x][q].y * w);
                    o[4 * q + 2] = fmaf(o[4 * q + 2], c, v[x][q].z * w);
                    o[4 * q + 3] = fmaf(o[4 * q + 3], c, v[x][q].w * w);
                }
            }
        }
        T* dst = static_cast<T*>(a.o) + ((size_t)cut.x * a.tokens + t) * a.n_heads * DH +
                 (size_t)(cut.y * n_rep + row - t_local * n_rep) * DH + cols * kJoinCols;
        store_joined(dst, o, 1.f / L);
    }
}

}  // namespace

}  // namespace llama
