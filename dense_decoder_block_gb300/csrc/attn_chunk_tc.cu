// Attention of chunks of new tokens over a paged cache on the tensor cores (bf16, head_dim 128).
//
// A tile is 256 query rows of a KV group (two halves of tqh tokens x the group's heads, 128 rows each), its keys come
// in chunks of 128:
//   S = Q K^T     tcgen05.mma M = N = K = 128, operands in shared memory
//   softmax       thread = row: a running reference m of the row (log2 domain), p = 2^(s c - m) rounded to bf16, l += the
//                 rounded p (in fp32), so that a weight's rounding goes to O and l alike: where one key outweighs the
//                 others, or the heavy ones hold one value, the row is that value.
//                 m follows the row's maximum only when that has grown by more than 2^kSlack, so O is
//                 seldom scaled (p <= 2^kSlack; nothing is lost, bf16 and fp32 keep their relative precision; a published
//                 technique of attention kernels)
//   O += P V      tcgen05.mma, P from tensor memory, O accumulated in tensor memory
// Two streams run side by side so that one's MMAs cover the other's softmax: the halves of a tile, or, when a tile has
// 128 rows at most (few new tokens), its even and its odd chunks, joined at the end.  A stream's S, P (over S) and O
// take 128 columns each for S and O.  Roles:
//   warp 0        Q, K and V: a page (at most 128 rows) is one TMA copy issued by a lane of its own, and lands as row
//                 groups of 8 with their two 64-column halves side by side (make_tmap_pages)
//   warps 1, 3    tensor memory, MMAs of stream 0, of stream 1: S, then PV when P is there, the first 64 keys ahead of
//                 the rest; whole warps, see umma_ss_warp
//   warp 2        the CTA's pieces (attn_chunk.cuh), a few ahead
//   warps 4..11   softmax of stream 0, of stream 1; scaling of O
//   warps 12..15  care of V, output
// Rows do not see what lies behind them: P is 0 there, and so that 0 times an infinity or a NaN does not reach
// O, such values of a tile's newest positions are taken out of the chunk's V and added to the rows that do see
// them at the end (an infinity or NaN in O either way).
//
// A piece of more than kTcCarry chunks goes through the pipeline in parts, each a softmax of its own: the output warps leave a
// part's O in the workspace and its (m, l) in shared memory, and take them into O of the next (attn_chunk.cuh says why;
// a carry within the softmax's loop cost every step 2 to 3 %; so: 9728 tokens of 4 / 1 heads behind 262144 3.00 -> 3.08 ms).
//
// Bound, over long rows, by the tensor pipe and what of a stream's softmax the other stream's MMAs do not cover: a chunk's
// four MMAs take 1.06 us, the step 1.45 (the pipe is 71 % active; the softmax issues in 50 % of the slots, at half the
// rate of ex2).  A tile costs 4 us beside its steps: the first copies, the first softmax, the output; a call 5 before its
// first MMA (lengths, the walk, the block table, Q and K: one load behind another).  Whole calls: 8192 tokens of 32 / 8
// heads 354 us on pages of 128 rows (1.55 PFLOP/s), 362 of 64, 385 of 16 (a copy a page); 4096 of 64 / 8 behind 4096 513
// (1.61) at 2070 MHz, 548 (1.51) once the power limit has taken the clock to 1920; 2048 of 32 / 8 42 to 46, 32 x 4 behind
// 1000 37.5 (3.5 TB/s), 100 behind 8192 34 (with the join), one token at 100 positions 7.6.
#include <algorithm>

#include "attn_chunk.cuh"
#include "attn_tc.cuh"

namespace llama {
namespace {

constexpr int kThreads = 512;
constexpr int kRegsCtrl = 72, kRegsSoftmax = 168, kRegsOut = 104;
constexpr int kRegsNeeded = 128 * kRegsCtrl + 256 * kRegsSoftmax + 128 * kRegsOut;
static_assert(kRegsNeeded <= 128 * kThreads, "register split exceeds the launch allocation");
constexpr float kSlack = 8.f;

constexpr int OFF_Q = 0;                      // [half] Q: 2 sub-tiles
constexpr int OFF_K = 4 * kSub;               // [stage] K, row groups of 8
constexpr int OFF_V = OFF_K + 4 * kSub;       // [stage] V
constexpr int OFF_BAR = OFF_V + 4 * kSub;
constexpr int OFF_PIECES = OFF_BAR + 512;     // the ring of pieces, and a word for each
constexpr int OFF_ML = OFF_PIECES + 256;      // [parity][stream][128] (m, l): see ml_full
constexpr int OFF_CARRY = OFF_ML + 4096;      // [half][128] (m, l) of the parts before
constexpr int OFF_SEQS = OFF_CARRY + 2048;
using Seqs = ChunkSeqs<kTcSeqs>;                 // of a launch
constexpr int SMEM_BYTES = OFF_SEQS + (int)sizeof(Seqs) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
constexpr int TM_S = 0, TM_O = 256;           // + 128 per stream

// A CTA's pieces as its roles read them: warp 2 walks the CTA's share a few pieces ahead and leaves them in a ring
// (a walk in every role took registers that the softmax does not have).
constexpr int kRing = 4;
static_assert(kRing * (sizeof(ChunkPiece) + sizeof(int)) <= 256, "ring entries");

// MMAs issued by a whole converged warp, one elected lane executing them.  With values that are
// uniform over the warp the compiler keeps descriptors in uniform registers, and an MMA costs the warp a few issue
// slots; from a branch that one lane takes it costs dozens, and a busy scheduler then holds the tensor cores back (S and PV of
// a 128-key chunk beside two warps of multiply-adds on the scheduler: 1025 cycles this way, 2080 the other).
__device__ __forceinline__ void umma_ss_warp(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_ts_warp(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_commit_warp(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(ptx::smem_u32(bar))
        : "memory");
}

// A page's rows, from row group `group` on (see make_tmap_pages), through the default policy: several tiles read them.
__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar, int group) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %3, %3, %4}], [%2];" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(0), "r"(group)
        : "memory");
}

// A barrier of n threads that tells whether `ok` holds for all of them.
__device__ __forceinline__ bool named_bar_and(int id, int n, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(n), "r"((uint32_t)ok)
        : "memory");
    return r != 0;
}

// The words of 2 bf16 whose exponent is all ones (infinity, NaN): bits 15 and 31.
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) { return ((w & 0x7fff7fffu) + 0x00800080u) & 0x80008000u; }

// Row `row` of a chunk's V, behind the tile's first position: cleared when it lies behind the last (it may hold
// anything), else its infinities and NaN are; true when there were any.  Rolled loops: it runs for one or two
// chunks of a tile.  (No call: a function of its own may use more registers than these warps keep.)
__device__ __forceinline__ bool care_for_v(uint8_t* v, int row, bool clear) {
    uint8_t* at = v + (row >> 3) * 2048 + (row & 7) * 128;
    uint32_t bad = 0;
#pragma unroll 2
    for (int i = 0; i < 16; ++i) {   // 16-byte columns in an order that spreads the rows over the banks
        uint4* u = reinterpret_cast<uint4*>(at + (i & 8) * 128 + ((i ^ row) & 7) * 16);
        if (clear) *u = make_uint4(0, 0, 0, 0);
        else bad |= not_finite2(u->x) | not_finite2(u->y) | not_finite2(u->z) | not_finite2(u->w);
    }
    if (!bad) return false;
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
        uint32_t* w = reinterpret_cast<uint32_t*>(at + (i >> 5) * 1024) + (i & 31);
        const uint32_t f = not_finite2(*w);
        *w &= ~((f & 0x8000u ? 0xffffu : 0u) | (f & 0x80000000u ? 0xffff0000u : 0u));
    }
    return true;
}

// A piece's steps: step i belongs to stream i % 2.  A pair (both halves have rows): both streams take every chunk.
// Else the streams take turns.
__device__ __forceinline__ bool is_pair(const ChunkPiece& p, int tqh) { return p.t1 - p.t0 > tqh; }
__device__ __forceinline__ int steps_of(const ChunkPiece& p, int tqh) { return (p.c1 - p.c0) << is_pair(p, tqh); }
__device__ __forceinline__ int steps_of_stream(const ChunkPiece& p, int tqh, int s) {
    const int n = p.c1 - p.c0;
    return is_pair(p, tqh) ? n : (n + 1 - s) >> 1;
}
// O of a row (its 128 columns in tensor memory, (m, l) = x) takes in what the parts before left at `carry`, (m, l) = y;
// returns (m, l) of both.  A side without a key above -inf has no weight, and 0 times its NaN is NaN.  The whole warp, two
// columns at a time: rarely called, and longer code slows all other tiles (sixteen: 8192 tokens 359 us, so 369).
__device__ __forceinline__ float2 take_in(uint32_t o_taddr, const float2& x, const float* carry, const float2& y) {
    const float m = fmaxf(x.x, y.x);
    const float wx = x.x == -INFINITY ? 0.f : ex2(x.x - m), wy = y.x == -INFINITY ? 0.f : ex2(y.x - m);
    auto load = [&](int cb) { return __ldcg(reinterpret_cast<const float2*>(carry + (cb >> 2) * 512 + (cb & 2))); };
    float2 next = load(0);
#pragma unroll 1
    for (int cb = 0; cb < 128; cb += 2) {
        float o[2];
        ptx::tmem_ld<2>(o_taddr + cb, o);
        const float2 before = next;
        next = load(min(cb + 2, 126));
        ptx::tmem_wait_ld();
        ptx::tmem_st2(o_taddr + cb, __fmaf_rn(before.x, wy, o[0] * wx), __fmaf_rn(before.y, wy, o[1] * wx));
    }
    ptx::tmem_wait_st();
    return make_float2(m, __fmaf_rn(y.y, wy, x.y * wx));
}
// The first chunk with keys behind the tile's first position: from here on V wants care.
__device__ __forceinline__ int care_from(const ChunkPiece& p) { return max(p.c0, (p.pos0 + 1) / kAttnChunk); }

__global__ void __launch_bounds__(kThreads, 1)
    k_attn_chunk(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                 const __grid_constant__ CUtensorMap mV, const ChunkArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = (uint64_t*)(sm + OFF_BAR);
    uint64_t* q_full = bars + 0;     // TMA -> MMA
    uint64_t* q_empty = bars + 1;    // MMA (both streams, after their last S of the piece) -> TMA
    uint64_t* k_full = bars + 2;     // [2] TMA -> MMA
    uint64_t* k_empty = bars + 4;    // [2] MMA (two arrivals: of each stream, or of the one that takes the chunk) -> TMA
    uint64_t* v_full = bars + 6;     // [2] TMA -> MMA
    uint64_t* v_empty = bars + 8;    // [2] MMA (as k_empty, after PV) -> TMA
    uint64_t* s_full = bars + 10;    // [stream] MMA -> softmax (S done, and PV of the step before)
    uint64_t* p_half = bars + 12;    // [stream] softmax (P of keys 0..63 written, O scaled) -> MMA
    uint64_t* p_full = bars + 14;    // [stream] softmax (the rest written) -> MMA
    uint64_t* care_req = bars + 16;  // [V stage] MMA (a chunk that wants care has landed) -> warps 12..15
    uint64_t* care_done = bars + 18; // [V stage] warps 12..15 -> MMA
    uint64_t* pv_done = bars + 20;   // [stream] MMA (after the last PV of a piece) -> warps 12..15
    // [parity][stream] softmax (m and l of the piece written) -> warps 12..15: the softmax may be through with
    // the stream's next piece (pieces it has steps of are counted) before they have looked at this one's
    uint64_t* ml_full = bars + 22;
    uint64_t* pc_full = bars + 26;   // [4] warp 2 -> all roles: piece j in entry j % 4
    // [4] -> warp 2: warps 12..15 (piece done), and MMA and softmax of stream 1 (entry read: they may have no step of
    // the piece; the other roles have read it when it is done)
    uint64_t* pc_free = bars + 30;
    uint64_t* o_free = bars + 34;    // [stream] warps 12..15 (O of a piece read) -> MMA
    uint64_t* lag = bars + 36;       // MMA of stream 0 -> MMA of stream 1: it may begin the piece
    uint32_t* tmem_holder = (uint32_t*)(bars + 37);
    ChunkPiece* pieces = (ChunkPiece*)(sm + OFF_PIECES);
    int* poison = (int*)(sm + OFF_PIECES + kRing * sizeof(ChunkPiece));   // [4] j + 1: care was taken of piece j's V
    Seqs& seqs = *reinterpret_cast<Seqs*>(sm + OFF_SEQS);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform
    ptx::griddep_wait();   // lengths, tables, rows: whatever the stream holds in front
    const int n_rep = a.n_heads / a.n_kv_heads, tqh = a.tq >> 1;
    int* err = a.err;

    if (threadIdx.x == 0) {
        ptx::mbar_init(q_full, 1);
        ptx::mbar_init(q_empty, 2);
        ptx::mbar_init(lag, 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&k_full[i], 1);
            ptx::mbar_init(&k_empty[i], 2);
            ptx::mbar_init(&v_full[i], 1);
            ptx::mbar_init(&v_empty[i], 2);
            ptx::mbar_init(&s_full[i], 1);
            ptx::mbar_init(&p_half[i], 4);
            ptx::mbar_init(&p_full[i], 4);
            ptx::mbar_init(&care_req[i], 1);
            ptx::mbar_init(&care_done[i], 4);
            ptx::mbar_init(&o_free[i], 4);
            ptx::mbar_init(&pv_done[i], 1);
            ptx::mbar_init(&ml_full[i], 4);
            ptx::mbar_init(&ml_full[2 + i], 4);
        }
        for (int i = 0; i < kRing; ++i) {
            ptx::mbar_init(&pc_full[i], 1);
            ptx::mbar_init(&pc_free[i], 9);
            poison[i] = 0;
        }
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_holder, 512);
        ptx::tmem_relinquish();
    }
    if (warp == 2) {
        chunk_seqs(a, seqs, blockIdx.x == 0);
        __syncwarp();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    // dependents start only once this CTA holds its tensor memory
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();

    // piece j, once it is there; false behind the last (or when a wait gave up)
    auto piece = [&](int j, ChunkPiece& p) -> bool {
        if (!ptx::mbar_wait(&pc_full[j % kRing], (j / kRing) & 1, err)) return false;
        p = pieces[j % kRing];
        return p.c0 < p.c1;
    };
    if (warp < 4) {
        ptx::setmaxnreg_dec<kRegsCtrl>();
        if (warp == 2) {
            // ------------------------------------------------------------------ the pieces
            ChunkWalk walk(a, seqs, blockIdx.x, gridDim.x);
            walk.begin(a);
            ChunkPiece p;
            p.c1 = p.to = 0;
            for (int j = 0;; ++j) {
                bool more = true;
                if (p.c1 < p.to) {
                    p.c0 = p.c1;   // the piece's next part
                } else {
                    more = walk.next(p);
                    p.from = p.c0;
                    p.to = p.c1;
                }
                p.c1 = min(p.to, p.c0 + kTcCarry);
                if (j >= kRing && !__all_sync(0xffffffffu, ptx::mbar_wait(&pc_free[j % kRing], ((j / kRing) & 1) ^ 1, err))) break;
                if (!more) p.c0 = p.c1 = p.to = 0;
                if (lane == 0) {
                    pieces[j % kRing] = p;
                    ptx::mbar_arrive(&pc_full[j % kRing]);
                }
                if (!more) break;
            }
        } else if (warp == 0) {
            // ------------------------------------------------------------------ TMA producer, the whole warp
            const int shift = a.pages.shift, ps = 1 << shift, box = min(ps, kAttnChunk);
            if (lane == 0) {
                ptx::prefetch_tmap(&mQ);
                ptx::prefetch_tmap(&mK);
                ptx::prefetch_tmap(&mV);
            }
            int kc = 0, vc = 0, n_q = 0;   // chunks of K and V, Q tiles issued
            bool ok = true;
            ChunkPiece p;
            // chunk c's copy into the next stage of a ring; lane = page of the chunk
            auto copy = [&](const CUtensorMap* map, int c, int id, int off, uint64_t* full, uint64_t* empty, int& gi) {
                const int st = gi & 1;
                int go = 1;
                if (lane == 0 && gi >= 2) go = ptx::mbar_wait(&empty[st], ((gi >> 1) & 1) ^ 1, err);
                ok = __shfl_sync(0xffffffffu, go, 0);
                if (!ok) return;
                const int n = (min(kAttnChunk, p.kv_last + 1 - c * kAttnChunk) + box - 1) / box;
                if (lane == 0) ptx::mbar_arrive_expect_tx(&full[st], n * box * 256);
                __syncwarp();
                if (lane < n) {
                    const int row = ((id * a.n_kv_heads + p.g) << shift) + (c * kAttnChunk & (ps - 1));
                    tma_load_page(sm + off + st * 2 * kSub + lane * box * 256, map, &full[st], row >> 3);
                }
                ++gi;
            };
            for (int j = 0; ok && piece(j, p); ++j) {
                // page ids are read a chunk ahead of their copies
                auto lookup = [&](int c) -> int {
                    if (c >= p.c1 || lane * box >= min(kAttnChunk, p.kv_last + 1 - c * kAttnChunk)) return 0;
                    const int id = page_of(a.pages, p.b, (c * kAttnChunk >> shift) + lane, err);
                    return max(id, 0);   // recorded; the rows are undefined, the copy stays inside the cache
                };
                int id = lookup(p.c0), before = 0;
                // Q's place is free when the piece before has its last S, K's a chunk earlier; the first piece waits for
                // its page ids
                if (j > 0) copy(&mK, p.c0, id, OFF_K, k_full, k_empty, kc);
                if (!ok) break;
                int go = 1;
                if (lane == 0 && j >= 1) go = ptx::mbar_wait(q_empty, (j - 1) & 1, err);
                if (!__shfl_sync(0xffffffffu, go, 0)) break;
                if (lane == 0) {
                    const int halves = is_pair(p, tqh) ? 2 : 1;
                    ptx::mbar_arrive_expect_tx(q_full, halves * 2 * n_rep * tqh * 128);
                    for (int x = 0; x < 2 * halves; ++x)
                        asm volatile(
                            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(ptx::smem_u32(sm + OFF_Q + x * kSub)),
                            "l"(reinterpret_cast<uint64_t>(&mQ)), "r"(ptx::smem_u32(q_full)), "r"((x & 1) * 64),
                            "r"(p.g * n_rep), "r"(p.b * a.tokens + p.t0 + (x >> 1) * tqh)
                            : "memory");
                }
                ++n_q;
                // K a chunk ahead of V: its stage is free earlier
                for (int c = p.c0; ok && c <= p.c1; ++c) {
                    const int next = lookup(c + 1);
                    if (c < p.c1 && (j == 0 || c > p.c0)) copy(&mK, c, id, OFF_K, k_full, k_empty, kc);
                    if (ok && c > p.c0) copy(&mV, c - 1, before, OFF_V, v_full, v_empty, vc);
                    before = id;
                    id = next;
                }
            }
            // no copy may still be landing when the CTA exits (it has landed already
            // unless a wait above gave up)
            if (lane == 0) {
                if (n_q > 0) ptx::mbar_wait_drain(q_full, (n_q - 1) & 1);
                for (int i = max(0, kc - 2); i < kc; ++i) ptx::mbar_wait_drain(&k_full[i & 1], (i >> 1) & 1);
                for (int i = max(0, vc - 2); i < vc; ++i) ptx::mbar_wait_drain(&v_full[i & 1], (i >> 1) & 1);
            }
        } else {
            // ------------------------------------------------------------------ MMA issuer of stream s, the whole warp
            // S(i + 1) follows PV(i) at once: MMAs run in issue order, so P(i) has been read when S(i + 1)
            // overwrites it, and the softmax has read S(i) before it wrote P(i).
            const int s = warp >> 1;
            auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
            const uint32_t s_tmem = tmem + TM_S + s * 128, o_tmem = tmem + TM_O + s * 128;
            const uint64_t k_desc = desc_with_stride(ptx::sw128_kmajor_desc(ptx::smem_u32(sm + OFF_K)), 2048);
            const uint64_t v_desc = desc_with_stride(ptx::sw128_mnmajor_desc(ptx::smem_u32(sm + OFF_V), 1024), 2048);
            int c0 = 0, step = 0;   // chunks of the pieces before, steps of the stream
            uint32_t cared = 0;     // parities of care_done
            bool ok = true;
            // every lane waits; the warp goes on or gives up as one
            auto wait = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, err)); };
            ChunkPiece p;
            for (int j = 0; ok && __all_sync(0xffffffffu, piece(j, p)); ++j) {
                const bool pair = uniform(is_pair(p, tqh));
                const int n = uniform(steps_of_stream(p, tqh, s)), chunks = uniform(p.c1 - p.c0);
                const int care = c0 + uniform(care_from(p) - p.c0);   // first chunk (counted as c) that wants care
                const uint64_t q_desc = ptx::sw128_kmajor_desc(ptx::smem_u32(sm + OFF_Q + (pair ? s : 0) * 2 * kSub));
                __syncwarp();
                if (s == 1 && lane == 0) ptx::mbar_arrive(&pc_free[j % kRing]);
                if (!wait(q_full, j & 1)) break;
                int c = c0 + (pair ? 0 : s);
                const int by = pair ? 1 : 2;
                // S of chunk c, the i-th of the piece
                auto issue_s = [&](int c, int i) -> bool {
                    const int st = c & 1;
                    if (!wait(&k_full[st], (c >> 1) & 1)) return false;
                    ptx::tc_fence_after();
                    const uint64_t k = k_desc + st * (2 * kSub / 16);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_ss_warp(s_tmem, q_desc + (ks / 4 * (kSub / 16) + ks % 4 * 2), k + (ks / 4 * 64 + ks % 4 * 2), IDESC_S,
                                     ks > 0);
                    umma_commit_warp(&s_full[s]);
                    umma_commit_warp(&k_empty[st]);
                    if (!pair) umma_commit_warp(&k_empty[st]);
                    if (i == n - 1) umma_commit_warp(q_empty);
                    return true;
                };
                // Streams that begin together stay together: their MMAs take turns, both then sit in their softmax and the
                // tensor cores are idle for it.  Stream 1 of a pair begins when stream 0 has its first P: from then on
                // the MMAs of one run under the softmax of the other (8192 tokens of 32 / 8 heads 450 -> 374 us, 4096
                // of 64 behind 4096 648 -> 532).  Streams that share a tile's chunks wait for copies instead.
                const bool together = !pair || n < 2;
                if (s == 0 && together && lane == 0) ptx::mbar_arrive(lag);
                if (s == 1 && !wait(lag, j & 1)) break;
                if (n > 0) {
                    ok = issue_s(c, 0);
                } else {   // no step of this piece (stream 1)
                    if (lane == 0) ptx::mbar_arrive(q_empty);
                    if (j > 0 && !wait(&o_free[s], (j - 1) & 1)) break;
                }
                for (int i = 0; ok && i < n; ++i, ++step, c += by) {
                    const int st = c & 1;
                    const uint64_t v = v_desc + st * (2 * kSub / 16);
                    // O of the last piece is read (and with that every chunk before is used, so that the
                    // parity of v_full tells this chunk's landing)
                    if (i == 0 && j > 0 && !wait(&o_free[s], (j - 1) & 1)) { ok = false; break; }
                    if (!wait(&v_full[st], (c >> 1) & 1)) { ok = false; break; }
                    if (c >= care) {
                        if ((!pair || s == 0) && lane == 0) ptx::mbar_arrive(&care_req[st]);
                        if (!wait(&care_done[st], cared >> st & 1)) { ok = false; break; }
                        cared ^= 1u << st;
                    }
                    if (!wait(&p_half[s], step & 1)) { ok = false; break; }
                    if (s == 0 && i == 0 && !together && lane == 0) ptx::mbar_arrive(lag);
                    ptx::tc_fence_after();
                    // P of keys 16ks.. in columns 8ks.., V rows 16ks..
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) umma_ts_warp(o_tmem, s_tmem + ks * 8, v + ks * 256, IDESC_PV, i > 0 || ks > 0);
                    if (!wait(&p_full[s], step & 1)) { ok = false; break; }
                    ptx::tc_fence_after();
#pragma unroll
                    for (int ks = 4; ks < 8; ++ks) umma_ts_warp(o_tmem, s_tmem + ks * 8, v + ks * 256, IDESC_PV, 1);
                    umma_commit_warp(&v_empty[st]);
                    if (!pair) umma_commit_warp(&v_empty[st]);
                    if (i == n - 1) umma_commit_warp(&pv_done[s]);
                    else ok = issue_s(c + by, i + 1);
                }
                // the other stream's chunks that want care, of which this one hears nothing
                if (!pair)
                    for (c = max(care, c0); c < c0 + chunks; ++c)
                        if (((c - c0) & 1) != s) cared ^= 1u << (c & 1);
                c0 += chunks;
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------------ softmax of a stream, thread = row
        ptx::setmaxnreg_inc<kRegsSoftmax>();
        const int s = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const int t_local = row / n_rep;
        const uint32_t s_taddr = tmem + ((uint32_t)(quarter * 32) << 16) + TM_S + s * 128;
        const uint32_t o_taddr = tmem + ((uint32_t)(quarter * 32) << 16) + TM_O + s * 128;
        const float c = a.scale_log2;
        int step = 0, took = 0;   // of the stream: steps, parity of its pieces
        bool ok = true;
        for (int j = 0;; ++j) {
            int left, last_key, ahead;   // chunks of the stream; the row's last key from the chunk's first; keys a step
            bool live;                   // rows in this quarter
            {
                ChunkPiece p;
                if (!piece(j, p)) break;
                const bool pair = is_pair(p, tqh);
                left = steps_of_stream(p, tqh, s);
                const int first = pair ? s * tqh : 0;   // token of the half
                const int rows = min(p.t1 - p.t0 - first, tqh) * n_rep;
                live = quarter * 32 < rows;
                ahead = pair ? kAttnChunk : 2 * kAttnChunk;
                __syncwarp();
                if (s == 1 && lane == 0) ptx::mbar_arrive(&pc_free[j % kRing]);
                last_key = row < rows ? p.pos0 + first + t_local - (p.c0 + (pair ? 0 : s)) * kAttnChunk : -1;
            }
            float m = -INFINITY, l = 0.f;
            const int steps = left;
#pragma unroll 1
            for (; left > 0; --left, ++step, last_key -= ahead) {
                if (ok) ok = ptx::mbar_wait(&s_full[s], step & 1, err);
                ptx::tc_fence_after();
                uint32_t weights[8][8];   // two rounded weights each
                float sc = 1.f;
                if (live) {
                    float v[128];
                    ptx::tmem_ld<32>(s_taddr, v);
                    ptx::tmem_ld<32>(s_taddr + 32, v + 32);
                    ptx::tmem_ld<32>(s_taddr + 64, v + 64);
                    ptx::tmem_ld<32>(s_taddr + 96, v + 96);
                    ptx::tmem_wait_ld();
                    if (!__all_sync(0xffffffffu, last_key >= kAttnChunk - 1)) {
#pragma unroll
                        for (int e0 = 0; e0 < 128; e0 += 32) {   // words of what is seen: bit e of the word is key e0 + e
                            const int over = 31 - (last_key - e0);
                            const uint32_t seen = over > 31 ? 0u : over <= 0 ? 0xffffffffu : 0xffffffffu >> over;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(seen >> e & 1)) v[e0 + e] = -INFINITY;
                        }
                    }
                    float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int e = 4; e < 124; e += 8) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) mx[x] = max3(mx[x], v[e + x], v[e + 4 + x]);
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) mx[x] = fmaxf(mx[x], v[124 + x]);
                    const float mn = fmaxf(m, __fmul_rn(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), c));
                    if (mn != m && !(mn - m <= kSlack)) {
                        sc = ex2(m - mn);
                        m = mn;
                    }
                    if (left < steps && __any_sync(0xffffffffu, sc != 1.f)) {
                        // O of the steps before (complete: see s_full); seldom after the first few
#pragma unroll 1
                        for (int cb = 0; cb < 128; cb += 16) {
                            float o[16];
                            ptx::tmem_ld<16>(o_taddr + cb, o);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= sc;
                            ptx::tmem_st16(o_taddr + cb, o);
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : m;
                    const uint64_t c2 = pack2(c, c), nm2 = pack2(-ref, -ref);
#pragma unroll
                    for (int e0 = 0; e0 < 128; e0 += 16) {
                        uint32_t (&packed)[8] = weights[e0 / 16];
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            float x0, x1, x2, x3;
                            unpack2(fma2(pack2(v[e0 + e], v[e0 + e + 1]), c2, nm2), x0, x1);
                            unpack2(fma2(pack2(v[e0 + e + 2], v[e0 + e + 3]), c2, nm2), x2, x3);
                            x0 = ex2(x0);
                            x1 = ex2(x1);
                            x2 = ex2(x2);
                            x3 = ex2(x3);
                            const __nv_bfloat162 p0 = __floats2bfloat162_rn(x0, x1), p1 = __floats2bfloat162_rn(x2, x3);
                            packed[e / 2] = *reinterpret_cast<const uint32_t*>(&p0);
                            packed[e / 2 + 1] = *reinterpret_cast<const uint32_t*>(&p1);
                        }
                        tmem_st8(s_taddr + e0 / 2, packed);
                        if (e0 == 48) {   // keys 0..63
                            ptx::tmem_wait_st();
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(&p_half[s]);
                        }
                    }
                    ptx::tmem_wait_st();
                } else if (lane == 0) {
                    ptx::mbar_arrive(&p_half[s]);
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&p_full[s]);
                // The rounded weights are summed while the MMAs have them (in front of the hand-over: 8192 tokens of 32 / 8
                // heads, 16-row pages 433 us, so 382; 4096 of 64 behind 4096 580 and 514).
                if (live) {
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < 64; e += 2) {
                        const uint32_t w0 = weights[e / 8][e % 8], w1 = weights[e / 8][e % 8 + 1];
                        sum[0] = add_bf16_lo(w0, sum[0]);
                        sum[1] = add_bf16_hi(w0, sum[1]);
                        sum[2] = add_bf16_lo(w1, sum[2]);
                        sum[3] = add_bf16_hi(w1, sum[3]);
                    }
                    l = __fmaf_rn(l, sc, (sum[0] + sum[2]) + (sum[1] + sum[3]));
                }
            }
            if (steps > 0) {
                reinterpret_cast<float2*>(sm + OFF_ML)[(took * 2 + s) * 128 + row] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&ml_full[took * 2 + s]);
                took ^= 1;
            }
        }
    } else {
        // ------------------------------------------------------------------ care of V, output
        ptx::setmaxnreg_dec<kRegsOut>();
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const int t_local = row / n_rep, h_local = row - t_local * n_rep;
        const uint32_t o_taddr = tmem + ((uint32_t)(quarter * 32) << 16) + TM_O;
        const float2* ml = reinterpret_cast<const float2*>(sm + OFF_ML) + row;
        float2* carried = reinterpret_cast<float2*>(sm + OFF_CARRY) + row;   // of this thread's rows
        bool ok = true;
        int c0 = 0;                        // chunks of the pieces before
        uint32_t took = 0, ml_phase = 0;   // parities of the streams' pieces, of ml_full
        uint32_t cared = 0;                // parities of care_req
        ChunkPiece p;
        for (int j = 0; named_bar_and(1, 128, piece(j, p)); ++j) {   // all four warps go on or none
            const bool pair = is_pair(p, tqh);
            const int steps = steps_of(p, tqh);
#pragma unroll 1
            for (int c = care_from(p); c < p.c1; ++c) {
                const int at = c0 + c - p.c0, v = at & 1, key = c * kAttnChunk + row;
                if (ok) ok = ptx::mbar_wait(&care_req[v], cared >> v & 1, err);
                if (ok) ok = ptx::mbar_wait(&v_full[v], (at >> 1) & 1, err);
                cared ^= 1u << v;
                if (key > p.pos0 && care_for_v(sm + OFF_V + v * 2 * kSub, row, key > p.kv_last)) poison[j % kRing] = j + 1;
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&care_done[v]);
            }
            c0 += p.c1 - p.c0;
            // output: the halves one after another, or the two streams of one half joined
            named_bar_and(1, 128, true);   // poison is written
            const bool poisoned = poison[j % kRing] == j + 1;
            const bool more = p.c1 < p.to;                       // parts behind this one
            const bool split = more || p.to - p.from < p.n;      // O and (m, l) are left as they are
            const int slot = 2 * blockIdx.x + (p.from == 0);
#pragma unroll 1
            for (int half = 0; half < (pair ? 2 : 1); ++half) {
                // this half's streams: `half`, or 0 and (with two chunks or more) 1
                const bool both = !pair && steps > 1;
                for (int s = half; s <= (both ? 1 : half); ++s) {
                    const int at = (took >> s & 1) * 2 + s;
                    if (ok) ok = ptx::mbar_wait(&ml_full[at], ml_phase >> at & 1, err);
                    ml_phase ^= 1u << at;
                    if (ok) ok = ptx::mbar_wait(&pv_done[s], took >> s & 1, err);
                }
                ptx::tc_fence_after();
                // O read: the next piece's first PV may overwrite it (half 0's while half 1 is stored)
                auto free_o = [&] {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::mbar_arrive(&o_free[half]);
                        if (!pair) ptx::mbar_arrive(&o_free[1]);
                    }
                };
                const int tokens = min(p.t1 - p.t0 - half * tqh, tqh);
                if (quarter * 32 >= tokens * n_rep) {
                    free_o();
                    continue;
                }
                const bool valid = t_local < tokens;
                float2 x = ml[((took >> half & 1) * 2 + half) * 128];
                float* carry = a.carry + (size_t)(2 * blockIdx.x + half) * (128 * 128) + row * 4;   // [column / 4][row][4]
                if (p.c0 > p.from) x = take_in(o_taddr + half * 128, x, carry, carried[half * 128]);
                float w0 = 1.f, w1 = 0.f;   // weights of the streams
                if (both) {
                    const float2 y = ml[((took >> 1) * 2 + 1) * 128];
                    // a stream without a key above -inf has no weight
                    const float M = fmaxf(x.x, y.x);
                    w0 = x.x == -INFINITY && x.y == 0.f ? 0.f : ex2(x.x - M);
                    w1 = y.x == -INFINITY && y.y == 0.f ? 0.f : ex2(y.x - M);
                    x = make_float2(M, __fmaf_rn(x.y, w0, y.y * w1));
                }
                bf16* dst = static_cast<bf16*>(a.o) + ((size_t)p.b * a.tokens + p.t0 + half * tqh + t_local) * a.n_heads * 128 +
                            (size_t)(p.g * n_rep + h_local) * 128;
                float* part = more ? carry : a.partial + (size_t)(2 * slot + half) * (128 * 128) + row * 4;
                if (more) {
                    carried[half * 128] = x;
                } else if (split) {
                    if (valid && ok) a.part_ml[(2 * slot + half) * 128 + row] = x;
                } else {
                    const float inv = __fdividef(1.f, x.y);   // no key above -inf: 0 * infinity
                    w0 *= inv;
                    w1 *= inv;
                }
#pragma unroll 1
                for (int cb = 0; cb < 128; cb += 32) {
                    float o[32];
                    ptx::tmem_ld<32>(o_taddr + half * 128 + cb, o);
                    if (both) {
                        float q[32];
                        ptx::tmem_ld<32>(o_taddr + 128 + cb, q);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __fmaf_rn(o[e], w0, q[e] * w1);
                    } else {
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e += 2) unpack2(mul2(pack2(o[e], o[e + 1]), pack2(w0, w0)), o[e], o[e + 1]);
                    }
                    if (!valid || !ok) {
                    } else if (split) {
#pragma unroll
                        for (int q4 = 0; q4 < 8; ++q4)
                            *reinterpret_cast<float4*>(part + (cb / 4 + q4) * 512) =
                                make_float4(o[4 * q4], o[4 * q4 + 1], o[4 * q4 + 2], o[4 * q4 + 3]);
                    } else {
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4) {
                            uint32_t packed[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 v2 = __floats2bfloat162_rn(o[8 * q4 + 2 * e], o[8 * q4 + 2 * e + 1]);
                                packed[e] = *reinterpret_cast<const uint32_t*>(&v2);
                            }
                            *reinterpret_cast<uint4*>(dst + cb + 8 * q4) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
                        }
                    }
                }
                free_o();
                if (poisoned && valid && ok) {
                    // infinities and NaN that were taken out of V: onto the columns of the rows that see them
                    const int first = max(p.pos0 + 1, p.c0 * kAttnChunk);
                    const int last = min(p.pos0 + half * tqh + t_local, p.c1 * kAttnChunk - 1);
                    for (int key = first; key <= last; ++key) {
                        const int id = max(page_of(a.pages, p.b, key >> a.pages.shift, nullptr), 0);
                        const size_t at = ((size_t)(id * a.n_kv_heads + p.g) << a.pages.shift) + (key & ((1 << a.pages.shift) - 1));
                        const bf16* v = static_cast<const bf16*>(a.vc) + at * 128;
                        for (int d = 0; d < 128; ++d) {
                            const float bad = __bfloat162float(v[d]);
                            if (bad - bad == 0.f) continue;
                            if (split) part[(d >> 2) * 512 + (d & 3)] += bad;
                            else dst[d] = __float2bfloat16_rn(__bfloat162float(dst[d]) + bad);
                        }
                    }
                }
            }
            took ^= steps > 1 ? 3 : 1;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&pc_free[j % kRing]);
        }
    }

    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_chunk_tc(const ChunkArgs& a, int head_dim, cudaStream_t s) {
    if (head_dim != 128) return cudaErrorInvalidValue;
    const int n_rep = a.n_heads / a.n_kv_heads, ps = 1 << a.pages.shift;
    const uint64_t rows = (uint64_t)a.pages.n_pages * a.n_kv_heads * ps;
    CUtensorMap mq, mk, mv;
    if (!make_tmap_pages(&mk, a.kc, rows, std::min(ps, kAttnChunk)) ||
        !make_tmap_pages(&mv, a.vc, rows, std::min(ps, kAttnChunk)))
        return cudaErrorInvalidValue;
    cudaError_t r = kernel_setup_once((const void*)k_attn_chunk, [](const void* kern) {
        // the register split inside the kernel must fit the block's launch allocation
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, kern);
        if (e != cudaSuccess) return e;
        if (fa.numRegs * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    });
    if (r != cudaSuccess) return r;
    for (int b0 = 0; b0 < a.batch; b0 += kTcSeqs) {
        ChunkArgs k = a;
        const size_t at = (size_t)b0 * a.tokens * a.n_heads * 128;
        k.batch = std::min(a.batch - b0, kTcSeqs);
        k.q = static_cast<const bf16*>(a.q) + at;
        k.o = static_cast<bf16*>(a.o) + at;
        k.start += b0;
        k.count += b0;
        k.pages.table += (size_t)b0 * a.pages.stride;
        if (!make_tmap_q3d(&mq, k.q, a.n_heads, k.batch * a.tokens, n_rep, k.tq / 2)) return cudaErrorInvalidValue;
        // persistent: one CTA per SM at most (work assigned on the device)
        const unsigned n_ctas = (unsigned)std::min(device_sm_count(), kTcCtas);
        r = launch_pdl(k_attn_chunk, dim3(n_ctas), dim3(kThreads), SMEM_BYTES, s, mq, mk, mv, k);
        if (r != cudaSuccess) return r;
        if (n_ctas == 1 || a.max_pos < kNeverSplit) continue;
        r = launch_pdl(k_attn_chunk_join<bf16, 128, 2, 128>, dim3(4 * n_ctas), dim3(kJoinThreads), 0, s, k, (int)n_ctas);
        if (r != cudaSuccess) return r;
    }
    return cudaSuccess;
}

}  // namespace llama
