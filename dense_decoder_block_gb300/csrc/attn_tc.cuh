// What the tensor-core attention kernels share: packed arithmetic, MMA chains, the prefill
// softmax, tensor maps.
#pragma once
#include <cudaTypedefs.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int kSub = 128 * 128;                 // one [128 rows][64 bf16] swizzled sub-tile, bytes
constexpr uint32_t IDESC_S = ptx::idesc_bf16_f32(128, 128);
constexpr uint32_t IDESC_PV = ptx::idesc_bf16_f32_bmn(128, 128);

// Byte offset of the 16-byte chunk `c16` (0..7) of row `r` in a 128-byte-swizzled sub-tile.
__device__ __forceinline__ uint32_t sw_off(int r, int c16) { return (uint32_t)(r * 128 + ((c16 ^ (r & 7)) << 4)); }

// 2^x on the special-function unit (PTX ex2.approx.ftz: max relative error
// 2^-22, far below the bf16 rounding of p that follows; results below the
// smallest normal float are flushed to zero).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 lanes in one 64-bit register pair, for the packed f32x2 arithmetic of
// sm_100 and later: each lane is the IEEE round-to-nearest operation of its scalar
// form (no flush to zero), so a packed result equals the two scalar results bit for
// bit -- it halves the instructions, not the precision.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {   // a * b + c, one rounding
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// acc + (the bf16 in the low / high half of p), exactly fadd(acc, float(half)):
// the mixed-precision add widens its bf16 operand exactly and rounds once.
__device__ __forceinline__ float add_bf16_lo(uint32_t p, float acc) {
    float r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tadd.rn.f32.bf16 %0, lo, %2;\n\t}"
        : "=f"(r) : "r"(p), "f"(acc));
    return r;
}
__device__ __forceinline__ float add_bf16_hi(uint32_t p, float acc) {
    float r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tadd.rn.f32.bf16 %0, hi, %2;\n\t}"
        : "=f"(r) : "r"(p), "f"(acc));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// max(a, b, c), exact like every max
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Eight 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Eight K = 16 steps of one accumulator chain from a single asm block.  Step ks's
// descriptors are step 0's plus the step's byte offset / 16 in the start-address
// field (shared-memory addresses stay below 256 KB, so the 14-bit field never
// carries: the same descriptors the per-step helpers build), the accumulate
// predicate off for step 0 and on after.  The issuing thread shares its scheduler
// with softmax and fold warps; this keeps its instructions per MMA few.
//
// Both operands from shared memory.  A is K-major in two 64-column sub-tiles
// A_SUB16 x 16 bytes apart (step ks at (ks / 4) sub-tiles + (ks % 4) * 32 bytes);
// B likewise with B_SUB16, or MN-major (B_MN: step ks 16 rows on, B_SUB16 x 16 bytes).
template <int A_SUB16, int B_SUB16, bool B_MN>
__device__ __forceinline__ void umma8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
#define LLAMA_AOFF(ks) ((ks) / 4 * A_SUB16 + (ks) % 4 * 2)
#define LLAMA_BOFF(ks) (B_MN ? (ks) * B_SUB16 : (ks) / 4 * B_SUB16 + (ks) % 4 * 2)
    asm volatile(
        "{\n\t.reg .pred pf, pt;\n\t.reg .b64 a<8>, b<8>;\n\t"
        "setp.ne.b32 pf, %3, %3;\n\tsetp.eq.b32 pt, %3, %3;\n\t"
        "add.s64 a1, %1, %4;\n\tadd.s64 b1, %2, %11;\n\t"
        "add.s64 a2, %1, %5;\n\tadd.s64 b2, %2, %12;\n\t"
        "add.s64 a3, %1, %6;\n\tadd.s64 b3, %2, %13;\n\t"
        "add.s64 a4, %1, %7;\n\tadd.s64 b4, %2, %14;\n\t"
        "add.s64 a5, %1, %8;\n\tadd.s64 b5, %2, %15;\n\t"
        "add.s64 a6, %1, %9;\n\tadd.s64 b6, %2, %16;\n\t"
        "add.s64 a7, %1, %10;\n\tadd.s64 b7, %2, %17;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pf;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a4, b4, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a5, b5, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a6, b6, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a7, b7, %3, pt;\n\t"
        "}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "n"(LLAMA_AOFF(1)), "n"(LLAMA_AOFF(2)), "n"(LLAMA_AOFF(3)), "n"(LLAMA_AOFF(4)), "n"(LLAMA_AOFF(5)),
        "n"(LLAMA_AOFF(6)), "n"(LLAMA_AOFF(7)), "n"(LLAMA_BOFF(1)), "n"(LLAMA_BOFF(2)), "n"(LLAMA_BOFF(3)),
        "n"(LLAMA_BOFF(4)), "n"(LLAMA_BOFF(5)), "n"(LLAMA_BOFF(6)), "n"(LLAMA_BOFF(7))
        : "memory");
#undef LLAMA_AOFF
#undef LLAMA_BOFF
}
// A from tensor memory (step ks 8 columns on: 16 bf16 per row), B MN-major from
// shared memory (step ks 16 rows = B_STEP16 x 16 bytes on).
template <int B_STEP16>
__device__ __forceinline__ void umma8_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred pf, pt;\n\t.reg .b32 t<8>;\n\t.reg .b64 b<8>;\n\t"
        "setp.ne.b32 pf, %3, %3;\n\tsetp.eq.b32 pt, %3, %3;\n\t"
        "add.u32 t1, %1, 8;\n\tadd.s64 b1, %2, %4;\n\t"
        "add.u32 t2, %1, 16;\n\tadd.s64 b2, %2, %5;\n\t"
        "add.u32 t3, %1, 24;\n\tadd.s64 b3, %2, %6;\n\t"
        "add.u32 t4, %1, 32;\n\tadd.s64 b4, %2, %7;\n\t"
        "add.u32 t5, %1, 40;\n\tadd.s64 b5, %2, %8;\n\t"
        "add.u32 t6, %1, 48;\n\tadd.s64 b6, %2, %9;\n\t"
        "add.u32 t7, %1, 56;\n\tadd.s64 b7, %2, %10;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, pf;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t1], b1, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t2], b2, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t3], b3, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t4], b4, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t5], b5, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t6], b6, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t7], b7, %3, pt;\n\t"
        "}"
        ::"r"(d), "r"(a_tmem), "l"(b), "r"(idesc), "n"(B_STEP16), "n"(2 * B_STEP16), "n"(3 * B_STEP16), "n"(4 * B_STEP16),
        "n"(5 * B_STEP16), "n"(6 * B_STEP16), "n"(7 * B_STEP16)
        : "memory");
}

// The same chains issued by a whole converged warp, one elected lane executing them.  With values that are
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

// The prefill softmax leaves P (bf16 pairs) in columns 0..63 of the S row and the row's (m, l) in
// columns 64, 65.
constexpr int PF_TM_ML = 64;

// Prefill softmax of one query row over one 128-key chunk, the keys split over
// two threads (two warps of the same TMEM lane quarter): half h holds keys
// 64h .. 64h+63 of the row's S in registers.  It computes exactly the canonical
// softmax: the row max over the visible keys is the max of the two halves' maxima
// (exchanged through shared memory; max is exact), p = bf16(2^(s c - m)) with
// hidden keys at -inf, and l = ((L0 + L1) + L2) + L3 with each quarter sum in
// ascending key order -- half 0 holds L0, L1, half 1 passes L2, L3 over.  Block c
// (keys 16c .. 16c+15) of P, packed as bf16 pairs, goes to columns 8c .. 8c+7 of
// the S row once both halves hold their scores in registers; half 0 writes the
// row's (m, l) to the ML columns.  `xch` is 4 x 128 floats of shared memory; `bar`
// the barrier id of this lane quarter.
__device__ __forceinline__ void softmax_half_tmem(uint32_t s_taddr, int h, int row, int jmax, float scale_log2,
                                                  float* xch, int bar, float& m_out) {
    float v[64];
    ptx::tmem_ld<32>(s_taddr + h * 64, v);
    ptx::tmem_ld<32>(s_taddr + h * 64 + 32, v + 32);
    ptx::tmem_wait_ld();
    const int jl = jmax - h * 64;   // last visible key of this half, local index
    const bool full = __all_sync(0xffffffffu, jl >= 63);
    float mx;
    if (full) {
        float a0 = v[0], a1 = v[1];
#pragma unroll
        for (int j = 2; j < 64; j += 4) {
            a0 = max3(a0, v[j], v[j + 1]);
            a1 = max3(a1, v[j + 2], v[j + 3]);
        }
        mx = fmaxf(a0, a1);
    } else {
        float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 64; ++j)
            if (j <= jl) a[j & 3] = fmaxf(a[j & 3], v[j]);
        mx = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
    }
    xch[h * 128 + row] = mx;
    ptx::named_bar_sync(bar, 64);   // both halves' maxima written, both S halves read
    const float m = __fmul_rn(fmaxf(xch[row], xch[128 + row]), scale_log2);
    const float m_use = (m != -INFINITY) ? m : 0.f;   // no visible key (or none above -inf): every p is 0
    if (!full) {
#pragma unroll
        for (int j = 0; j < 64; ++j)
            if (j > jl) v[j] = -INFINITY;
    }
    // The two quarter sums of this half (blocks 0, 1: quarter 2h; blocks 2, 3:
    // quarter 2h + 1) advance side by side, each in ascending key order, each
    // rounded p added straight from its bf16 half.
    const uint64_t c2 = pack2(scale_log2, scale_log2), nm2 = pack2(-m_use, -m_use);
    float lq[2] = {0.f, 0.f};
#pragma unroll
    for (int cp = 0; cp < 2; ++cp) {   // blocks cp (keys 64h + 16cp ..) and cp + 2
        const float* va = v + cp * 16;
        const float* vb = v + (cp + 2) * 16;
        uint32_t pa[8], pb[8];
#pragma unroll
        for (int t = 0; t < 16; t += 2) {
            float xa0, xa1, xb0, xb1;
            unpack2(fma2(pack2(va[t], va[t + 1]), c2, nm2), xa0, xa1);
            unpack2(fma2(pack2(vb[t], vb[t + 1]), c2, nm2), xb0, xb1);
            const __nv_bfloat162 ba = __floats2bfloat162_rn(ex2(xa0), ex2(xa1));
            const __nv_bfloat162 bb = __floats2bfloat162_rn(ex2(xb0), ex2(xb1));
            pa[t >> 1] = *reinterpret_cast<const uint32_t*>(&ba);
            pb[t >> 1] = *reinterpret_cast<const uint32_t*>(&bb);
            lq[0] = add_bf16_hi(pa[t >> 1], add_bf16_lo(pa[t >> 1], lq[0]));
            lq[1] = add_bf16_hi(pb[t >> 1], add_bf16_lo(pb[t >> 1], lq[1]));
        }
        tmem_st8(s_taddr + (h * 4 + cp) * 8, pa);
        tmem_st8(s_taddr + (h * 4 + cp + 2) * 8, pb);
    }
    if (h == 1) {
        xch[256 + row] = lq[0];
        xch[384 + row] = lq[1];
    }
    ptx::named_bar_sync(bar, 64);   // L2, L3 written; the maxima read
    if (h == 0) {
        const float l = __fadd_rn(__fadd_rn(__fadd_rn(lq[0], lq[1]), xch[256 + row]), xch[384 + row]);
        ptx::tmem_st2(s_taddr + PF_TM_ML, m, l);
    }
    ptx::tmem_wait_st();
    m_out = m;
}

// A page's rows, from row group `group` on (see make_tmap_pages).
__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar, int group, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %3, %3, %4}], [%2], %5;" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(0), "r"(group), "l"(policy)
        : "memory");
}

// The same through the default policy: rows that several tiles read.
__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar, int group) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %3, %3, %4}], [%2];" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(0), "r"(group)
        : "memory");
}

// A descriptor's distance between 8-row groups (stride byte offset) set to `bytes`.
__device__ __forceinline__ uint64_t desc_with_stride(uint64_t desc, uint32_t bytes) {
    return (desc & ~(0x3FFFull << 32)) | ((uint64_t)(bytes >> 4) << 32);
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
    if (!f) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &qr) !=
                cudaSuccess ||
            qr != cudaDriverEntryPointSuccess)
            return nullptr;
        f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        fn.store(f, std::memory_order_release);
    }
    return f;
}

// A paged K or V cache, `rows` rows of 128 bf16, as [rows / 8][2][8][64]; box: `box_rows` rows.
inline bool make_tmap_pages(CUtensorMap* map, const void* base, uint64_t rows, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {64, 8, 2, rows / 8};
    cuuint64_t strides[3] = {128 * 2, 64 * 2, 8 * 128 * 2};
    cuuint32_t box[4] = {64, 8, 2, (cuuint32_t)box_rows / 8};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool make_tmap_q3d(CUtensorMap* map, const void* q, int n_heads, int tokens, int n_rep, int tq) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {128, (cuuint64_t)n_heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {128 * 2, (cuuint64_t)n_heads * 128 * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)n_rep, (cuuint32_t)tq};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace llama
