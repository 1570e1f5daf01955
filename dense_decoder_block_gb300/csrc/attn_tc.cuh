// What the tensor-core attention kernels share: packed and mixed arithmetic, tensor maps.
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
