// Attention of chunks of new tokens over a paged cache on the tensor cores (bf16, head_dim 128).
//
// Tiles, chunks, softmax and fold are those of the contiguous prefill kernel (attn_tc.cu): 128 query rows
// (tq tokens x the heads of a KV group) against 128-key chunks in ascending order, S and O_c = P V by
// tcgen05.mma with the operands in shared and tensor memory, softmax weights rounded to bf16, O folded
// in fp32 registers.  A tile that one CTA walks from its first chunk to its last has the bits of the
// contiguous prefill's rows.  What differs:
//   - a chunk's rows lie in pages: a page (at most 128 rows) is one TMA copy issued by a lane of its own, and
//     lands as row groups of 8 with their two 64-column halves side by side (see make_tmap_pages);
//   - sequences have starts and counts of their own, read on the device (attn_chunk.cuh), and long caches under
//     few rows are split over the CTAs;
//   - rows do not see what lies behind them: P is 0 there, and so that 0 times an infinity or a NaN does not reach
//     O, such values of a tile's newest positions are taken out of the chunk's V and added to the
//     rows that do see them at the end (an infinity or NaN in O either way);
//   - 32-row quarters of a tile without a row (short chunks) skip the softmax and the fold.
#include <algorithm>

#include "attn_chunk.cuh"
#include "attn_tc.cuh"

namespace llama {
namespace {

constexpr int kThreads = 512;
// register split (launch: 128 per thread): as in the contiguous prefill, the fold threads hold a row of O each
constexpr int kRegsCtrl = 56;
constexpr int kRegsSoftmax = 112;
constexpr int kRegsFold = 232;
constexpr int kRegsNeeded = 128 * kRegsCtrl + 256 * kRegsSoftmax + 128 * kRegsFold;
static_assert(kRegsNeeded <= 128 * kThreads, "register split exceeds the launch allocation");
constexpr int OFF_Q = 0;                      // [buffer] Q: 2 sub-tiles
constexpr int OFF_K = 4 * kSub;               // [stage] K, row groups of 8
constexpr int OFF_V = OFF_K + 4 * kSub;       // [stage] V
constexpr int OFF_BAR = OFF_V + 4 * kSub;
constexpr int OFF_XCH = OFF_BAR + 256;        // softmax halves' exchange: 4 x 128 floats
constexpr int OFF_SEQS = OFF_XCH + 2048;
constexpr int SMEM_BYTES = OFF_SEQS + (int)sizeof(ChunkSeqs) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
static_assert(sizeof(ChunkSeqs) % 8 == 0 && OFF_SEQS % 8 == 0, "alignment of the prefix sums");
constexpr int kSBufs = 3;                     // S[i % 3] at columns 0 / 128 / 256, O_c at 384
constexpr int TM_S = 0, TM_OC = 384;

// The words of 2 bf16 whose exponent is all ones (infinity, NaN): bits 15 and 31.
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) { return ((w & 0x7fff7fffu) + 0x00800080u) & 0x80008000u; }

__global__ void __launch_bounds__(kThreads, 1)
    k_attn_chunk(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                 const __grid_constant__ CUtensorMap mV, const ChunkArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = (uint64_t*)(sm + OFF_BAR);
    uint64_t* q_full = bars + 0;     // [2] TMA -> MMA (the Q tile of this CTA's piece j in buffer j % 2)
    uint64_t* q_empty = bars + 2;    // [2] MMA (after the piece's last S) -> TMA
    uint64_t* k_full = bars + 4;     // [2] TMA -> MMA
    uint64_t* k_empty = bars + 6;    // [2] MMA (after S) -> TMA
    uint64_t* v_full = bars + 8;     // [2] TMA -> MMA (and the softmax, before it clears rows)
    uint64_t* v_empty = bars + 10;   // [2] MMA (after PV) -> TMA
    uint64_t* s_full = bars + 12;    // [3] MMA (after S) -> softmax
    uint64_t* p_full = bars + 15;    // [3] softmax (P, m, l written) -> MMA, fold
    uint64_t* s_free = bars + 18;    // [3] fold (m, l read) -> MMA
    uint64_t* oc_full = bars + 21;   // MMA (after PV) -> fold
    uint64_t* oc_free = bars + 22;   // fold (O_c read) -> MMA
    uint32_t* tmem_holder = (uint32_t*)(bars + 23);
    int* poison = (int*)(bars + 24); // [4] j + 1: piece j has infinities or NaN among its newest values
    ChunkSeqs& seqs = *reinterpret_cast<ChunkSeqs*>(sm + OFF_SEQS);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::griddep_wait();   // lengths, tables, rows: whatever the stream holds in front
    const int n_rep = a.n_heads / a.n_kv_heads;
    const int n_ctas = gridDim.x;
    int* err = a.err;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&q_full[i], 1);
            ptx::mbar_init(&q_empty[i], 1);
            ptx::mbar_init(&k_full[i], 1);
            ptx::mbar_init(&k_empty[i], 1);
            ptx::mbar_init(&v_full[i], 1);
            ptx::mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kSBufs; ++i) {
            ptx::mbar_init(&s_full[i], 1);
            ptx::mbar_init(&p_full[i], 8);
            ptx::mbar_init(&s_free[i], 4);
        }
        ptx::mbar_init(oc_full, 1);
        ptx::mbar_init(oc_free, 4);
        ptx::fence_mbar_init();
        for (int i = 0; i < 4; ++i) poison[i] = 0;
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_holder, 512);
        ptx::tmem_relinquish();
    }
    if (warp == 2) chunk_seqs(a, seqs, blockIdx.x == 0);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // dependents start only once this CTA holds its tensor memory
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();

    if (warp < 4) {
        ptx::setmaxnreg_dec<kRegsCtrl>();
        if (warp == 0 || warp == 2) {
            // ------------------------------------------------------------------ TMA producers (K and Q, V), whole warps
            const bool is_k = (warp == 0);
            const CUtensorMap* map = is_k ? &mK : &mV;
            uint64_t* full = is_k ? k_full : v_full;
            uint64_t* empty = is_k ? k_empty : v_empty;
            uint8_t* ring = sm + (is_k ? OFF_K : OFF_V);
            const int shift = a.pages.shift, ps = 1 << shift, box = min(ps, kAttnChunk);
            const uint64_t pol = ptx::policy_evict_last();   // the tiles of a KV head read the same rows
            if (lane == 0) ptx::prefetch_tmap(map);
            int gi = 0, n_q = 0;   // chunks and Q tiles issued
            bool ok = true;
            ChunkWalk walk(a, seqs, blockIdx.x, n_ctas);
            ChunkPiece p;
            for (int j = 0; ok && walk.next(p); ++j) {
                // lane = page of a chunk: its id is read a chunk ahead of its copy
                auto pages_in = [&](int c) { return (min(kAttnChunk, p.kv_last + 1 - c * kAttnChunk) + box - 1) / box; };
                auto lookup = [&](int c) -> int {
                    if (c >= p.c1 || lane >= pages_in(c)) return 0;
                    const int id = page_of(a.pages, p.b, (c * kAttnChunk >> shift) + lane, is_k ? err : nullptr);
                    return max(id, 0);   // recorded; the rows are undefined, the copy stays inside the cache
                };
                int next = lookup(p.c0);
                if (is_k) {
                    // Q of piece j into buffer j % 2 once piece j - 2's S MMAs are done with it
                    const int qb = j & 1;
                    int go = 1;
                    if (lane == 0 && j >= 2) go = ptx::mbar_wait(&q_empty[qb], ((j >> 1) - 1) & 1, err);
                    if (!__shfl_sync(0xffffffffu, go, 0)) { ok = false; break; }
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(&q_full[qb], 2 * n_rep * a.tq * 128);
                        for (int half = 0; half < 2; ++half)
                            asm volatile(
                                "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                                " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
                                    ptx::smem_u32(sm + OFF_Q + qb * 2 * kSub + half * kSub)),
                                "l"(reinterpret_cast<uint64_t>(&mQ)), "r"(ptx::smem_u32(&q_full[qb])), "r"(half * 64),
                                "r"(p.g * n_rep), "r"(p.b * a.tokens + p.t0)
                                : "memory");
                    }
                    ++n_q;
                }
                for (int c = p.c0; c < p.c1; ++c, ++gi) {
                    const int st = gi & 1;
                    int go = 1;
                    if (lane == 0 && gi >= 2) go = ptx::mbar_wait(&empty[st], ((gi >> 1) & 1) ^ 1, err);
                    if (!__shfl_sync(0xffffffffu, go, 0)) { ok = false; break; }
                    const int n = pages_in(c), id = next;
                    if (lane == 0) ptx::mbar_arrive_expect_tx(&full[st], n * box * 256);
                    __syncwarp();
                    if (lane < n) {
                        const int row = ((id * a.n_kv_heads + p.g) << shift) + (c * kAttnChunk & (ps - 1));
                        tma_load_page(ring + st * 2 * kSub + lane * box * 256, map, &full[st], row >> 3, pol);
                    }
                    next = lookup(c + 1);
                }
            }
            // no copy may still be landing when the CTA exits (it has landed already
            // unless a wait above gave up)
            if (lane == 0) {
                for (int j = max(0, n_q - 2); j < n_q; ++j) ptx::mbar_wait_drain(&q_full[j & 1], (j >> 1) & 1);
                for (int i = max(0, gi - 2); i < gi; ++i) ptx::mbar_wait_drain(&full[i & 1], (i >> 1) & 1);
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------------ MMA issuer
            if (lane == 0) {
                // S(gi) into S[gi % 3]: Q of its piece landed (at the piece's first chunk),
                // K(gi) landed, and the fold has read chunk gi - 3's (m, l) from that buffer
                // (PV(gi - 3), which read its P, was issued before and the MMAs run in issue
                // order).  After a piece's last S its Q buffer is released.
                ChunkWalk walk(a, seqs, blockIdx.x, n_ctas);
                ChunkPiece p;
                int s_j = 0, s_left = 0, issued = 0;   // piece of the next S, chunks left of it, S issued
                bool first = true;
                s_left = walk.next(p) ? p.c1 - p.c0 : 0;
                auto issue_s = [&]() -> bool {
                    if (s_left == 0) return true;
                    const int gi = issued, k = gi & 1, sb = gi % kSBufs, qb = s_j & 1;
                    if (first && !ptx::mbar_wait(&q_full[qb], (s_j >> 1) & 1, err)) return false;
                    if (!ptx::mbar_wait(&k_full[k], (gi >> 1) & 1, err)) return false;
                    if (gi >= kSBufs && !ptx::mbar_wait(&s_free[sb], ((gi / kSBufs) & 1) ^ 1, err)) return false;
                    ptx::tc_fence_after();
                    const uint64_t q_desc = ptx::sw128_kmajor_desc(ptx::smem_u32(sm + OFF_Q + qb * 2 * kSub));
                    const uint32_t k_addr = ptx::smem_u32(sm + OFF_K + k * 2 * kSub);
                    umma8_ss<kSub / 16, 1024 / 16, false>(tmem + TM_S + sb * 128, q_desc,
                                                          desc_with_stride(ptx::sw128_kmajor_desc(k_addr), 2048), IDESC_S);
                    ptx::umma_commit(&s_full[sb]);
                    ptx::umma_commit(&k_empty[k]);
                    ++issued;
                    first = false;
                    if (--s_left == 0) {
                        ptx::umma_commit(&q_empty[qb]);
                        ++s_j;
                        first = true;
                        s_left = walk.next(p) ? p.c1 - p.c0 : 0;
                    }
                    return true;
                };
                bool ok = true;
                for (int i = 0; i < kSBufs && ok; ++i) ok = issue_s();
                for (int gi = 0; ok && gi < issued; ++gi) {
                    const int k = gi & 1, sb = gi % kSBufs;
                    if (!ptx::mbar_wait(&p_full[sb], (gi / kSBufs) & 1, err)) break;
                    // O_c is overwritten once the fold has read chunk gi - 1's
                    if (gi >= 1 && !ptx::mbar_wait(oc_free, (gi - 1) & 1, err)) break;
                    if (!ptx::mbar_wait(&v_full[k], (gi >> 1) & 1, err)) break;
                    ptx::tc_fence_after();
                    const uint32_t v_addr = ptx::smem_u32(sm + OFF_V + k * 2 * kSub);
                    // P of keys 16ks.. in TMEM columns 8ks.., V rows 16ks..
                    umma8_ts<256>(tmem + TM_OC, tmem + TM_S + sb * 128,
                                  desc_with_stride(ptx::sw128_mnmajor_desc(v_addr, 1024), 2048), IDESC_PV);
                    ptx::umma_commit(oc_full);
                    ptx::umma_commit(&v_empty[k]);
                    ok = issue_s();
                }
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------------ softmax, two threads per row
        ptx::setmaxnreg_dec<kRegsSoftmax>();
        const int h = (warp - 4) >> 2;   // key half of this warpgroup
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        const int t_local = row / n_rep;
        float* xch = reinterpret_cast<float*>(sm + OFF_XCH);
        bool ok = true;
        int gi = 0;
        ChunkWalk walk(a, seqs, blockIdx.x, n_ctas);
        ChunkPiece p;
        for (int j = 0; walk.next(p); ++j) {
            const bool live = quarter * 32 < (p.t1 - p.t0) * n_rep;   // rows in this quarter
            const bool valid = p.t0 + t_local < p.t1 && t_local < a.tq;
            const int pos_r = p.pos0 + t_local;
            for (int c = p.c0; c < p.c1; ++c, ++gi) {
                const int k = gi & 1, sb = gi % kSBufs;
                // s_full(gi) also means PV(gi - 3) -- issued before S(gi) -- is done with the P in S[sb]
                if (ok) ok = ptx::mbar_wait(&s_full[sb], (gi / kSBufs) & 1, err);
                ptx::tc_fence_after();
                const int jmax = valid ? min(kAttnChunk - 1, pos_r - c * kAttnChunk) : -1;
                float m;
                // both halves reach the two barriers inside on every chunk, whatever `ok` says
                if (live)
                    softmax_half_tmem(tmem + lane_addr + TM_S + sb * 128, h, row, jmax, a.scale_log2, xch, 1 + quarter, m);
                if (h == 0) {
                    // values behind the first row: those past the tile's last position may hold anything and
                    // are cleared, infinities and NaN among those that only some rows see are taken out
                    // (P is 0 where they are hidden and 0 * NaN would poison O)
                    if (c * kAttnChunk + kAttnChunk - 1 > p.pos0) {
                        if (ok) ok = ptx::mbar_wait(&v_full[k], (gi >> 1) & 1, err);
                        const int key = c * kAttnChunk + row;
                        uint8_t* vrow = sm + OFF_V + k * 2 * kSub + (row >> 3) * 2048 + (row & 7) * 128;
                        if (key > p.kv_last) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int c16 = (i ^ (row & 7)) * 16;   // spread over the banks
                                *reinterpret_cast<uint4*>(vrow + c16) = make_uint4(0, 0, 0, 0);
                                *reinterpret_cast<uint4*>(vrow + 1024 + c16) = make_uint4(0, 0, 0, 0);
                            }
                        } else if (key > p.pos0) {
                            uint32_t bad = 0;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const uint4 u = *reinterpret_cast<const uint4*>(vrow + (i & 8) * 128 + ((i ^ row) & 7) * 16);
                                bad |= not_finite2(u.x) | not_finite2(u.y) | not_finite2(u.z) | not_finite2(u.w);
                            }
                            if (bad) {
                                poison[j & 3] = j + 1;
#pragma unroll 1
                                for (int i = 0; i < 64; ++i) {
                                    uint32_t* at = reinterpret_cast<uint32_t*>(vrow + (i >> 5) * 1024) + (i & 31);
                                    const uint32_t f = not_finite2(*at);
                                    *at &= ~((f & 0x8000u ? 0xffffu : 0u) | (f & 0x80000000u ? 0xffff0000u : 0u));
                                }
                            }
                        }
                    }
                    ptx::fence_proxy_async_smem();
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&p_full[sb]);
            }
        }
    } else {
        // ------------------------------------------------------------------ fold + output
        ptx::setmaxnreg_inc<kRegsFold>();
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        const int t_local = row / n_rep, h_local = row - t_local * n_rep;
        float O[128];
        bool ok = true;
        int gi = 0;
        ChunkWalk walk(a, seqs, blockIdx.x, n_ctas);
        if (threadIdx.x == kThreads - 1) a.cuts[blockIdx.x] = walk.begin();
        ChunkPiece p;
        for (int j = 0; walk.next(p); ++j) {
            const bool live = quarter * 32 < (p.t1 - p.t0) * n_rep;
            const bool valid = p.t0 + t_local < p.t1 && t_local < a.tq;
            float M = -INFINITY, L_sum = 0.f;
            bool started = false;
#pragma unroll 1
            for (int c = p.c0; c < p.c1; ++c, ++gi) {
                const int sb = gi % kSBufs;
                if (ok) ok = ptx::mbar_wait(&p_full[sb], (gi / kSBufs) & 1, err);
                ptx::tc_fence_after();
                float ml[2] = {-INFINITY, 0.f};
                if (live) {
                    ptx::tmem_ld<2>(tmem + lane_addr + TM_S + sb * 128 + PF_TM_ML, ml);
                    ptx::tmem_wait_ld();
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&s_free[sb]);
                const float m = ml[0], l = ml[1];
                if (ok) ok = ptx::mbar_wait(oc_full, gi & 1, err);
                ptx::tc_fence_after();
                if (!live) {
                    if (lane == 0) ptx::mbar_arrive(oc_free);
                    continue;
                }
                // Per row: skip a chunk with no visible key (or none above -inf), start from the first
                // one, fold the rest.  The TMEM loads are issued by the whole
                // warp whatever each row does (they are warp-collective).
                const bool use = !(m == -INFINITY && l == 0.f);
                const bool fold = use && started;
                float alpha = 1.f, beta = 0.f;
                if (fold) {
                    const float Mn = fmaxf(M, m);
                    alpha = exp2f(__fsub_rn(M, Mn));
                    beta = exp2f(__fsub_rn(m, Mn));
                    L_sum = __fmaf_rn(L_sum, alpha, __fmul_rn(l, beta));
                    M = Mn;
                } else if (use) {
                    M = m;
                    L_sum = l;
                }
                const uint32_t oc_addr = tmem + lane_addr + TM_OC;
#pragma unroll
                for (int cb = 0; cb < 4; ++cb) {
                    float oc[32];
                    ptx::tmem_ld<32>(oc_addr + cb * 32, oc);
                    ptx::tmem_wait_ld();
                    if (cb == 3) {   // O_c fully read: PV(gi + 1) may overwrite it
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(oc_free);
                    }
                    if (fold) {   // o = fma(o, alpha, oc * beta), two columns per instruction
                        const uint64_t a2 = pack2(alpha, alpha), b2 = pack2(beta, beta);
#pragma unroll
                        for (int jj = 0; jj < 32; jj += 2) {
                            float& o0 = O[cb * 32 + jj];
                            float& o1 = O[cb * 32 + jj + 1];
                            unpack2(fma2(pack2(o0, o1), a2, mul2(pack2(oc[jj], oc[jj + 1]), b2)), o0, o1);
                        }
                    } else if (use) {
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) O[cb * 32 + jj] = oc[jj];
                    }
                }
                started = started || use;
            }
            if (!started) {   // no key above -inf: nothing of a split row, NaN (0 / 0) for a whole one
                L_sum = 0.f;
#pragma unroll
                for (int jj = 0; jj < 128; ++jj) O[jj] = 0.f;
            }
            if (!valid || !ok) continue;
            bf16* dst = static_cast<bf16*>(a.o) + ((size_t)p.b * a.tokens + p.t0 + t_local) * a.n_heads * 128 +
                        (size_t)(p.g * n_rep + h_local) * 128;
            const bool split = p.c1 - p.c0 < p.n;
            const int slot = 2 * blockIdx.x + (p.c0 == 0);
            float* part = a.partial + (size_t)slot * (128 * 128) + row * 4;   // [column / 4][row][4]
            if (split) {
                a.part_ml[slot * 128 + row] = make_float2(M, L_sum);
#pragma unroll
                for (int d4 = 0; d4 < 32; ++d4)
                    *reinterpret_cast<float4*>(part + d4 * 512) =
                        make_float4(O[4 * d4], O[4 * d4 + 1], O[4 * d4 + 2], O[4 * d4 + 3]);
            } else {
                // o = O * (1 / L), rounded to bf16, while the next piece's chunks run
                const float inv_l = __frcp_rn(L_sum);
#pragma unroll
                for (int c8 = 0; c8 < 16; ++c8) {
                    uint32_t packed[4];
#pragma unroll
                    for (int jj = 0; jj < 8; jj += 2) {
                        const __nv_bfloat162 v2 = __floats2bfloat162_rn(__fmul_rn(O[c8 * 8 + jj], inv_l),
                                                                        __fmul_rn(O[c8 * 8 + jj + 1], inv_l));
                        packed[jj >> 1] = *reinterpret_cast<const uint32_t*>(&v2);
                    }
                    *reinterpret_cast<uint4*>(dst + c8 * 8) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
                }
            }
            if (poison[j & 3] == j + 1) {
                // infinities and NaN that the softmax warps took out of V: onto the columns of the rows that see them
                const int first = max(p.pos0 + 1, p.c0 * kAttnChunk);
                const int last = min(min(p.pos0 + t_local, p.kv_last), p.c1 * kAttnChunk - 1);
                for (int key = first; key <= last; ++key) {
                    const int id = max(page_of(a.pages, p.b, key >> a.pages.shift, nullptr), 0);
                    const size_t at = ((size_t)(id * a.n_kv_heads + p.g) << a.pages.shift) + (key & ((1 << a.pages.shift) - 1));
                    const bf16* v = static_cast<const bf16*>(a.vc) + at * 128;
                    for (int d = 0; d < 128; ++d) {
                        const float x = __bfloat162float(v[d]);
                        if (x - x == 0.f) continue;
                        if (split) part[(d >> 2) * 512 + (d & 3)] += x;
                        else dst[d] = __float2bfloat16_rn(__bfloat162float(dst[d]) + x);
                    }
                }
            }
        }
    }

    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Joins the pieces of a split tile: CTA (i, part of the columns), i the first CTA that begins inside the tile.
// Pieces in ascending order: o = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p, M the largest m_p.
constexpr int kJoinCols = 16;

__global__ void __launch_bounds__(128) k_attn_chunk_join(const ChunkArgs a, int n_ctas) {
    ptx::griddep_wait();
    const int i = blockIdx.x + 1, row = threadIdx.x;
    const int4 cut = __ldcg(a.cuts + i), before = __ldcg(a.cuts + i - 1);
    auto same = [&](const int4& x) { return x.w > 0 && x.x == cut.x && x.y == cut.y && x.z == cut.z; };
    if (cut.w == 0 || same(before)) return;
    const int n_rep = a.n_heads / a.n_kv_heads;
    const int t_local = row / n_rep, t = cut.z * a.tq + t_local;
    const bool valid = t_local < a.tq && t < a.count[cut.x];
    // the pieces: CTA i - 1's last, then the first ones of CTAs i, i + 1, ... (empty where the next begins at the
    // same chunk)
    float M = -INFINITY, L = 0.f;
    float o[kJoinCols];
#pragma unroll
    for (int e = 0; e < kJoinCols; ++e) o[e] = 0.f;
    auto add = [&](int slot) {
        const float2 ml = __ldcg(a.part_ml + slot * 128 + row);
        if (!valid || (ml.x == -INFINITY && ml.y == 0.f)) return;
        const float Mn = fmaxf(M, ml.x);
        const float c = M == -INFINITY ? 0.f : exp2f(M - Mn), w = exp2f(ml.x - Mn);
        M = Mn;
        L = fmaf(L, c, ml.y * w);
        const float4* part = reinterpret_cast<const float4*>(a.partial + (size_t)slot * (128 * 128)) + row;
#pragma unroll
        for (int q = 0; q < kJoinCols / 4; ++q) {
            const float4 v = __ldcg(part + (blockIdx.y * (kJoinCols / 4) + q) * 128);
            o[4 * q] = fmaf(o[4 * q], c, v.x * w);
            o[4 * q + 1] = fmaf(o[4 * q + 1], c, v.y * w);
            o[4 * q + 2] = fmaf(o[4 * q + 2], c, v.z * w);
            o[4 * q + 3] = fmaf(o[4 * q + 3], c, v.w * w);
        }
    };
    add(2 * (i - 1) + 1);
    int4 at = cut;
    for (int j = i; j < n_ctas; ++j) {
        const int4 next = j + 1 < n_ctas ? __ldcg(a.cuts + j + 1) : make_int4(0, 0, 0, 0);
        const bool more = same(next);
        if (!more || next.w > at.w) add(2 * j);
        if (!more) break;
        at = next;
    }
    if (!valid) return;
    bf16* dst = static_cast<bf16*>(a.o) + ((size_t)cut.x * a.tokens + t) * a.n_heads * 128 +
                (size_t)(cut.y * n_rep + row - t_local * n_rep) * 128 + blockIdx.y * kJoinCols;
    const float inv = 1.f / L;
#pragma unroll
    for (int e = 0; e < kJoinCols; e += 8) {
        uint32_t packed[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const __nv_bfloat162 v2 = __floats2bfloat162_rn(o[e + 2 * q] * inv, o[e + 2 * q + 1] * inv);
            packed[q] = *reinterpret_cast<const uint32_t*>(&v2);
        }
        *reinterpret_cast<uint4*>(dst + e) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
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
    for (int b0 = 0; b0 < a.batch; b0 += kChunkSeqs) {
        ChunkArgs k = a;
        const size_t at = (size_t)b0 * a.tokens * a.n_heads * 128;
        k.batch = std::min(a.batch - b0, kChunkSeqs);
        k.q = static_cast<const bf16*>(a.q) + at;
        k.o = static_cast<bf16*>(a.o) + at;
        k.start += b0;
        k.count += b0;
        k.pages.table += (size_t)b0 * a.pages.stride;
        if (!make_tmap_q3d(&mq, k.q, a.n_heads, k.batch * a.tokens, n_rep, a.tq)) return cudaErrorInvalidValue;
        // persistent: one CTA per SM at most (stretches of work assigned on the device)
        const unsigned n_ctas = (unsigned)std::min(device_sm_count(), kChunkMaxCtas / 2);
        r = launch_pdl(k_attn_chunk, dim3(n_ctas), dim3(kThreads), SMEM_BYTES, s, mq, mk, mv, k);
        if (r != cudaSuccess) return r;
        if (a.whole || n_ctas == 1) continue;
        r = launch_pdl(k_attn_chunk_join, dim3(n_ctas - 1, 128 / kJoinCols), dim3(128), 0, s, k, (int)n_ctas);
        if (r != cudaSuccess) return r;
    }
    return cudaSuccess;
}

}  // namespace llama
