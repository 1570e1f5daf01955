// Addressing of a paged KV cache, shared by the kernels that read and write it.
//
// K and V are [n_pages, n_kv_heads, page_size, head_dim]: the block's cache layout
// with a page in the place of a sequence.  Position p of sequence b lies in row
// p % page_size of page table[b][p / page_size]; page sizes are powers of two, so
// both are a shift and a mask.  Every page id read from a table is checked against
// [0, n_pages) before it becomes an address; offsets in elements are 64-bit.
#pragma once
#include "common.cuh"

namespace llama {

struct PageTable {
    const int* table = nullptr;   // [sequences][stride]
    int stride = 0;
    int n_pages = 0;
    int shift = 0;                // log2(page_size)
};

// Page `j` of sequence b, or -1 (recorded) when the entry is no page of the cache.
__device__ __forceinline__ int page_of(const PageTable& t, int b, int j, int* err) {
    const int id = t.table[(size_t)b * t.stride + j];
    if (id >= 0 && id < t.n_pages) return id;
    record_error(err, LLAMA_ERR_INVALID_ARG);
    return -1;
}

// Keys that sequence b attends in a call whose position word is `v` (`off` = 0: the
// sequence's position, v + 1 keys; off = -1: the number of keys itself, which may be
// 0).  0 for a word out of range; `bad` reports that.
__device__ __forceinline__ int paged_keys(int v, int off, int max_pos, bool& bad) {
    const long long p = (long long)v + off;
    bad = p >= max_pos || p < off;
    return bad ? 0 : (int)(p + 1);
}

inline bool page_size_ok(int ps) { return ps >= 16 && ps <= 1024 && (ps & (ps - 1)) == 0; }
inline int page_shift(int ps) {
    int s = 0;
    while ((1 << s) < ps) ++s;
    return s;
}

}  // namespace llama
