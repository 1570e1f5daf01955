// Paged KV cache: block tables and slot maps built on the device, prefilled rows
// stored into pages, and the reordering of beams' tables and unfilled pages.
//
// All kernels are launched with programmatic stream serialization, wait for the
// kernels before them before they read anything, and let their dependents start
// only when they end: the step's attention reads tables and older cache rows ahead
// of its own wait, so nothing that writes those may still be running by then.
#include <algorithm>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace llama {
namespace {

// ----------------------------------------------------------------------------- plan and release
// Request b holds ceil(start / ps) pages and needs ceil((start + count) / ps); the
// difference f_b is taken from the top of the free stack (plan) or given back
// (release), in the order of requests and of pages within a request:
//   o_b = f_0 + ... + f_{b-1},   page i of request b's fresh pages <-> stack entry
//   n_free - 1 - (o_b + i) (plan), n_free + F - 1 - (o_b + i) (release, F = sum f),
// so a release undoes the plan of the same requests exactly.
//
// One launch, no CTA waits on another: every CTA scans all requests (8 bytes each,
// from L2) for the prefix sums it needs and takes a contiguous run of the items --
// tokens of the slot map [batch][tokens], or table entries [batch][stride].  The
// CTA that handles a fresh page's first token also writes that page's table entry.
// Which CTA may write the new count: of one CTA, that one; into other words than it is read
// from, the first; in place under several CTAs none, since another may still be to read it:
// k_paged_count follows.  (A ticket word beside the count could tell the last CTA, but only
// where it was zero before the call.)  A million slots (256 requests of up to 4096 tokens) take
// 6.4 us, one CTA's chain of round trips 4.7; the call's host side 12.
constexpr int kPlanThreads = 256;
constexpr int kPlanItems = 8 * kPlanThreads;   // items per CTA

struct PlanArgs {
    const int* start;
    const int* count;
    int batch, width;        // items per request: tokens (plan) or table columns (release)
    int tokens;              // plan: columns of the slot map (counts above it are refused); release: INT_MAX
    int shift, n_pages;
    int* free_pages;         // [n_pages]
    const int* pool;         // {free pages, not read}
    int* pool_out;
    bool write_count;        // this launch writes pool_out
    int* table;
    int stride;
    int* slots;              // plan
    int* err;
};

// The pages request b takes: false (none) when its words are out of range.
__device__ __forceinline__ bool request_pages(const PlanArgs& a, int b, int& start, int& count, int& held, int& fresh) {
    start = __ldcg(a.start + b);
    count = __ldcg(a.count + b);
    const long long end = (long long)start + count, ps = 1ll << a.shift;
    const bool ok = start >= 0 && count >= 0 && count <= a.tokens && end <= INT32_MAX &&
                    end <= (long long)a.stride << a.shift;
    held = ok ? (int)((start + ps - 1) >> a.shift) : 0;
    fresh = ok ? (int)((end + ps - 1) >> a.shift) - held : 0;
    return ok;
}

__device__ __forceinline__ void write_pool(const PlanArgs& a, int n_free, long long moved, bool release) {
    a.pool_out[0] = (int)(n_free + (release ? moved : -moved));
    a.pool_out[1] = 0;
}

template <bool RELEASE>
__global__ void __launch_bounds__(kPlanThreads) k_paged_plan(const PlanArgs a) {
    __shared__ int s_start[kPlanItems + 2], s_count[kPlanItems + 2], s_off[kPlanItems + 2];   // requests of this CTA
    __shared__ long long s_warp[kPlanThreads / 32];
    __shared__ int s_free;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ptx::griddep_wait();
    if (tid == 0) s_free = __ldcg(a.pool);
    const long long n_items = RELEASE || a.tokens > 0 ? (long long)a.batch * a.width : 0;   // no slots: the requests are checked alone
    const long long i0 = (long long)blockIdx.x * kPlanItems;
    const long long i1 = i0 + kPlanItems < n_items ? i0 + kPlanItems : n_items;
    const int b_lo = i1 > i0 ? (int)(i0 / a.width) : 0;
    const int b_hi = i1 > i0 ? (int)((i1 - 1) / a.width) : -1;   // at most kPlanItems requests apart

    // prefix sums of the fresh pages over all requests (64-bit: a sum beyond any pool
    // must not wrap into one that fits)
    long long total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int start = 0, count = 0, held = 0, fresh = 0;
        if (b < a.batch && !request_pages(a, b, start, count, held, fresh)) {
            count = -1;   // no slots, no pages
            if (blockIdx.x == 0) record_error(a.err, LLAMA_ERR_POS_RANGE);
        }
        long long x = fresh;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        long long before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            const long long v = s_warp[w];
            before += w < warp ? v : 0;
            all += v;
        }
        if (b >= b_lo && b <= b_hi) {
            s_start[b - b_lo] = start;
            s_count[b - b_lo] = count;
            s_off[b - b_lo] = (int)min(total + before + x - fresh, (long long)INT32_MAX);
        }
        total += all;
        __syncthreads();
    }
    if (a.batch == 0) __syncthreads();   // (the scan above has barriers of its own)
    const int n_free = s_free;
    const bool pool_ok = n_free >= 0 && n_free <= a.n_pages;
    const bool enough = pool_ok && (RELEASE ? total <= a.n_pages - n_free : total <= n_free);
    if (!enough && blockIdx.x == 0 && tid == 0) record_error(a.err, pool_ok ? LLAMA_ERR_NO_PAGES : LLAMA_ERR_INVALID_ARG);

    const int mask = (1 << a.shift) - 1;
    int i0_done = 0;   // items handled in runs
    const unsigned before = (unsigned)(i0 - (long long)b_lo * a.width);   // items of b_lo before this CTA's
    if constexpr (!RELEASE) {
        // Rows of 8 tokens or more: a thread takes 8 consecutive slots, which lie in a page or
        // two of a request or two, and stores them as two vectors (one slot per thread and
        // turn: 9.5 us for a million slots).
        constexpr int kRun = kPlanItems / kPlanThreads;
        const int n = (int)(i1 - i0) - tid * kRun;
        if (a.width >= kRun && n >= kRun && ((uintptr_t)a.slots & 15) == 0) {
            const unsigned x = before + tid * kRun;
            unsigned q = x / (unsigned)a.width;
            int t = (int)(x - q * (unsigned)a.width), start = 0, count = -1, off = 0, held = 0, page = -1, id = -1;
            bool fresh = true;   // a new request
            int slot[kRun];
#pragma unroll
            for (int e = 0; e < kRun; ++e, ++t) {
                if (t == a.width) {
                    t = 0;
                    ++q;
                    fresh = true;
                }
                if (fresh) {
                    start = s_start[q];
                    count = s_count[q];
                    off = s_off[q];
                    held = (int)(((long long)start + mask) >> a.shift);
                    page = -1;
                    fresh = false;
                }
                slot[e] = -1;
                if (!enough || t >= count) continue;
                const int pos = start + t, j = pos >> a.shift;
                int* entry = a.table + (size_t)(b_lo + (int)q) * a.stride + j;
                if (j != page) {
                    page = j;
                    id = __ldcg(j < held ? entry : a.free_pages + (n_free - 1 - (off + (j - held))));
                    if (id < 0 || id >= a.n_pages) record_error(a.err, LLAMA_ERR_INVALID_ARG);
                }
                if (j >= held && (pos & mask) == 0) *entry = id;
                if (id >= 0 && id < a.n_pages) slot[e] = (id << a.shift) + (pos & mask);
            }
            int4* to = reinterpret_cast<int4*>(a.slots + i0 + tid * kRun);
            to[0] = make_int4(slot[0], slot[1], slot[2], slot[3]);
            to[1] = make_int4(slot[4], slot[5], slot[6], slot[7]);
            static_assert(kRun == 8, "two vectors");
        }
        if (a.width >= kRun && ((uintptr_t)a.slots & 15) == 0) {
            // what is left of the last CTA's items, below one thread's run
            i0_done = (int)(i1 - i0) / kRun * kRun;
        }
    }
#pragma unroll 4
    for (int e = i0_done + tid; e < (int)(i1 - i0); e += kPlanThreads) {
        const unsigned x = before + e, q = x / (unsigned)a.width;
        const int b = b_lo + (int)q, t = (int)(x - q * (unsigned)a.width);
        const int start = s_start[q], count = s_count[q], off = s_off[q];
        const int held = (int)(((long long)start + mask) >> a.shift);
        if constexpr (RELEASE) {
            const int need = (int)(((long long)start + count + mask) >> a.shift);
            if (enough && count >= 0 && t >= held && t < need) {
                const int id = __ldcg(a.table + (size_t)b * a.stride + t);
                if (id < 0 || id >= a.n_pages) record_error(a.err, LLAMA_ERR_INVALID_ARG);
                a.free_pages[n_free + total - 1 - (off + (t - held))] = id;
            }
        } else {
            int slot = -1;
            if (enough && t < count) {
                const int pos = start + t, j = pos >> a.shift;
                const int id = __ldcg(j < held ? a.table + (size_t)b * a.stride + j
                                               : a.free_pages + (n_free - 1 - (off + (j - held))));
                if (j >= held && (pos & mask) == 0) a.table[(size_t)b * a.stride + j] = id;
                if (id >= 0 && id < a.n_pages) slot = (id << a.shift) + (pos & mask);
                else record_error(a.err, LLAMA_ERR_INVALID_ARG);
            }
            a.slots[i0 + e] = slot;
        }
    }
    if (a.write_count && blockIdx.x == 0 && tid == 0) write_pool(a, n_free, enough ? total : 0, RELEASE);
}

// The new count in place, behind a plan or release of several CTAs: the same sum, the same
// conditions (recorded there).
template <bool RELEASE>
__global__ void __launch_bounds__(kPlanThreads) k_paged_count(const PlanArgs a) {
    __shared__ unsigned long long s_total;
    const int tid = threadIdx.x;
    ptx::griddep_wait();
    if (tid == 0) s_total = 0;
    __syncthreads();
    unsigned long long mine = 0;
    for (int b = tid; b < a.batch; b += kPlanThreads) {
        int start, count, held, fresh;
        request_pages(a, b, start, count, held, fresh);
        mine += fresh;
    }
    atomicAdd(&s_total, mine);
    __syncthreads();
    if (tid > 0) return;
    const int n_free = __ldcg(a.pool);
    const long long total = (long long)s_total;
    const bool enough = n_free >= 0 && n_free <= a.n_pages && (RELEASE ? total <= a.n_pages - n_free : total <= n_free);
    write_pool(a, n_free, enough ? total : 0, RELEASE);
}

// ----------------------------------------------------------------------------- store
// Row copies: token t of sequence b, source row src_pos + t of every KV head, goes to
// slot s = slots[b][t]: page s / page_size, row s % page_size.  A negative slot is
// skipped.  Bound by the copy's bytes; a thread moves kStoreVec 16-byte vectors of K
// and of V, all loads issued before the stores.
constexpr int kStoreThreads = 256;
constexpr int kStoreVec = 4;

struct StoreArgs {
    const uint4* k;
    const uint4* v;
    uint4* pk;
    uint4* pv;
    const int* slots;
    int tokens, src_seq, src_pos, n_kv_heads, shift, log_vec;   // 2^log_vec vectors per row
    long long n_slots;
    int* err;
};

__global__ void __launch_bounds__(kStoreThreads) k_paged_store(const StoreArgs a) {
    ptx::griddep_wait();
    const int g = blockIdx.y, b = blockIdx.z;
    const size_t src0 = (((size_t)b * a.n_kv_heads + g) * a.src_seq + a.src_pos) << a.log_vec;
    const long long n = (long long)a.tokens << a.log_vec;
    const long long first = (long long)blockIdx.x * (kStoreThreads * kStoreVec) + threadIdx.x;
    uint4 k[kStoreVec], v[kStoreVec];
    long long dst[kStoreVec];
#pragma unroll
    for (int i = 0; i < kStoreVec; ++i) {
        const long long x = first + i * kStoreThreads;
        dst[i] = -1;
        if (x < n) {
            const int t = (int)(x >> a.log_vec);
            const int s = __ldcg(a.slots + (size_t)b * a.tokens + t);
            if (s >= a.n_slots) record_error(a.err, LLAMA_ERR_INVALID_ARG);
            if (s >= 0 && s < a.n_slots) {
                const long long row = (((long long)(s >> a.shift) * a.n_kv_heads + g) << a.shift) + (s & ((1 << a.shift) - 1));
                dst[i] = (row << a.log_vec) + (x & ((1 << a.log_vec) - 1));
                k[i] = __ldcg(a.k + src0 + x);
                v[i] = __ldcg(a.v + src0 + x);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kStoreVec; ++i)
        if (dst[i] >= 0) {
            a.pk[dst[i]] = k[i];
            a.pv[dst[i]] = v[i];
        }
}

// ----------------------------------------------------------------------------- beam reorder
// Rows g * beams .. g * beams + beams - 1 are the beams of request g, all of the same
// length: c full pages and r rows of page c, which each beam owns.  Beam i continues
// parent p(i): its first c table entries become p(i)'s (full pages are never written
// again, so beams share them) and rows 0..r-1 of its own page c become those of p(i)'s
// page c, in every layer.
//
// A CTA per (layer, K or V, request, part of a page): reading the lengths, parents and pages
// again for each costs less than a CTA walking several layers, whose copies then wait for
// one another (31 us against 34 for 8 requests of 4 beams, 28 rows in 32 layers; 156 MB).
//
// In place without a copy of the state: a thread owns one 16-byte column (layer, K or
// V, head, row, vector) of the unfilled page across all beams, or one table column,
// reads it for every beam that changes and only then writes.  Any map of parents,
// swaps included, is therefore safe, and no thread waits on another.
constexpr int kReorderThreads = 256;
constexpr int kReorderLayers = 128;   // layers per launch (their pointers are kernel arguments)
constexpr int kMaxBeams = 32;

struct ReorderArgs {
    const int* parents;
    const int* lens;
    int* table;
    int beams, stride, shift, n_pages, n_kv_heads, log_vec, n_layers;
    bool move_table;
    int* err;
    uint4* kv[2 * kReorderLayers];   // K and V of each layer
};

template <int B>
__global__ void __launch_bounds__(kReorderThreads) k_beam_reorder(const __grid_constant__ ReorderArgs a) {
    __shared__ int s_par[kMaxBeams], s_page[kMaxBeams];
    __shared__ int s_bad;
    const int tid = threadIdx.x, g = blockIdx.z;
    const size_t row0 = (size_t)g * a.beams;
    ptx::griddep_wait();
    if (tid == 0) s_bad = 0;
    __syncthreads();
    const int len = __ldcg(a.lens + row0);
    const bool len_ok = len >= 0 && len <= (long long)a.stride << a.shift;
    const int c = len_ok ? len >> a.shift : 0, r = len_ok ? len & ((1 << a.shift) - 1) : 0;
    if (tid < a.beams) {
        const long long p = (long long)a.parents[row0 + tid] - (long long)row0;
        const int page = r > 0 ? a.table[(row0 + tid) * a.stride + c] : 0;
        if (p < 0 || p >= a.beams || !len_ok || a.lens[row0 + tid] != len || page < 0 || page >= a.n_pages) s_bad = 1;
        s_par[tid] = (int)p;
        s_page[tid] = page;
    }
    __syncthreads();
    if (tid < a.beams && r > 0)   // a page that two beams would fill cannot be copied in place
        for (int i = 0; i < tid; ++i)
            if (s_page[i] == s_page[tid]) s_bad = 1;
    __syncthreads();
    if (s_bad) {   // the whole group stays as it was
        if (tid == 0) record_error(a.err, LLAMA_ERR_INVALID_ARG);
        return;
    }
    if ((int)blockIdx.y == 2 * a.n_layers) {   // table columns
        for (int j = blockIdx.x * kReorderThreads + tid; j < c; j += gridDim.x * kReorderThreads) {
            int v[B];
#pragma unroll
            for (int i = 0; i < B; ++i)
                if (i < a.beams && s_par[i] != i) v[i] = __ldcg(a.table + (row0 + s_par[i]) * a.stride + j);
#pragma unroll
            for (int i = 0; i < B; ++i)
                if (i < a.beams && s_par[i] != i) a.table[(row0 + i) * a.stride + j] = v[i];
        }
        return;
    }
    uint4* kv = a.kv[blockIdx.y];
    const int n = (a.n_kv_heads * r) << a.log_vec;
    for (int x = blockIdx.x * kReorderThreads + tid; x < n; x += gridDim.x * kReorderThreads) {
        const int hr = x >> a.log_vec, h = hr / r, t = hr - h * r;
        const size_t in = ((((size_t)h << a.shift) + t) << a.log_vec) + (x & ((1 << a.log_vec) - 1));
        const size_t page = (size_t)a.n_kv_heads << (a.shift + a.log_vec);
        uint4 v[B];
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (i < a.beams && s_par[i] != i) v[i] = __ldcg(kv + s_page[s_par[i]] * page + in);
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (i < a.beams && s_par[i] != i) kv[s_page[i] * page + in] = v[i];
    }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// 16-byte vectors of a row (log2), or -1 for a type and head size the cache does not take.
int row_log_vec(int head_dim, int dtype) {
    if (dtype == LLAMA_BF16) return head_dim == 128 ? 4 : -1;
    if (dtype != LLAMA_F32) return -1;
    return head_dim == 32 ? 3 : head_dim == 64 ? 4 : head_dim == 128 ? 5 : -1;
}

int check_geometry(int page_size, int n_pages) {
    if (n_pages <= 0) return LLAMA_ERR_INVALID_ARG;
    if (!page_size_ok(page_size)) return LLAMA_ERR_UNSUPPORTED_DIMS;
    // slots are int32
    if ((long long)n_pages * page_size > INT32_MAX) return LLAMA_ERR_UNSUPPORTED_DIMS;
    return LLAMA_OK;
}

}  // namespace

int paged_cache_check(const llama_paged_cache* kv, int n_kv_heads, int head_dim, int dtype) {
    if (!kv || !kv->k || !kv->v || !aligned16(kv->k) || !aligned16(kv->v)) return LLAMA_ERR_INVALID_ARG;
    if (dtype != LLAMA_BF16 && dtype != LLAMA_F32) return LLAMA_ERR_INVALID_ARG;
    if (n_kv_heads <= 0) return LLAMA_ERR_INVALID_ARG;
    if (row_log_vec(head_dim, dtype) < 0) return LLAMA_ERR_UNSUPPORTED_DIMS;
    const int rc = check_geometry(kv->page_size, kv->n_pages);
    if (rc != LLAMA_OK) return rc;
    // rows of the cache are addressed by int32 coordinates (TMA) and the heads by a grid dimension
    if (n_kv_heads > 65535 || (long long)kv->n_pages * kv->page_size * n_kv_heads > INT32_MAX)
        return LLAMA_ERR_UNSUPPORTED_DIMS;
    return LLAMA_OK;
}

}  // namespace llama

using namespace llama;

namespace {

template <bool RELEASE>
int run_plan(PlanArgs a, cudaStream_t s) {
    const long long items = (long long)a.batch * a.width;
    const long long ctas = std::max<long long>(1, (items + kPlanItems - 1) / kPlanItems);
    if (ctas > INT32_MAX) return LLAMA_ERR_INVALID_ARG;
    a.write_count = ctas == 1 || a.pool_out != a.pool;
    cudaError_t e = launch_pdl(k_paged_plan<RELEASE>, dim3((unsigned)ctas), dim3(kPlanThreads), 0, s, a);
    if (e == cudaSuccess && !a.write_count) e = launch_pdl(k_paged_count<RELEASE>, dim3(1), dim3(kPlanThreads), 0, s, a);
    return e == cudaSuccess ? LLAMA_OK : LLAMA_ERR_CUDA;
}

// The pool's two words, in place or apart: not one word's overlap of a pool that is read and one
// that is written.
bool pools_ok(const int32_t* pool, const int32_t* pool_out) {
    if (!pool || !pool_out) return false;
    const uintptr_t p = (uintptr_t)pool, q = (uintptr_t)pool_out;
    return p == q || (p > q ? p - q : q - p) >= 2 * sizeof(int32_t);
}

}  // namespace

extern "C" int llama_paged_plan(const int32_t* start, const int32_t* count, int batch, int tokens, int page_size,
                                int n_pages, const int32_t* free_pages, const int32_t* pool, int32_t* pool_out,
                                int32_t* table, int table_stride, int32_t* slots, int32_t* err_dev, void* stream) {
    if (batch < 0 || tokens < 0 || table_stride <= 0) return LLAMA_ERR_INVALID_ARG;
    const int rc = check_geometry(page_size, n_pages);
    if (rc != LLAMA_OK) return rc;
    if (!pools_ok(pool, pool_out)) return LLAMA_ERR_INVALID_ARG;
    if (batch > 0 && (!start || !count || !free_pages || !table || (tokens > 0 && !slots))) return LLAMA_ERR_INVALID_ARG;
    PlanArgs a{};
    a.start = start;
    a.count = count;
    a.batch = batch;
    a.width = std::max(tokens, 1);
    a.tokens = tokens;
    a.shift = page_shift(page_size);
    a.n_pages = n_pages;
    a.free_pages = const_cast<int32_t*>(free_pages);
    a.pool = pool;
    a.pool_out = pool_out;
    a.table = table;
    a.stride = table_stride;
    a.slots = slots;
    a.err = err_dev;
    return run_plan<false>(a, (cudaStream_t)stream);
}

extern "C" int llama_paged_release(const int32_t* start, const int32_t* count, int batch, int page_size, int n_pages,
                                   int32_t* free_pages, const int32_t* pool, int32_t* pool_out, const int32_t* table,
                                   int table_stride, int32_t* err_dev, void* stream) {
    if (batch < 0 || table_stride <= 0) return LLAMA_ERR_INVALID_ARG;
    const int rc = check_geometry(page_size, n_pages);
    if (rc != LLAMA_OK) return rc;
    if (!pools_ok(pool, pool_out)) return LLAMA_ERR_INVALID_ARG;
    if (batch > 0 && (!start || !count || !free_pages || !table)) return LLAMA_ERR_INVALID_ARG;
    PlanArgs a{};
    a.start = start;
    a.count = count;
    a.batch = batch;
    a.width = table_stride;
    a.tokens = INT32_MAX;
    a.shift = page_shift(page_size);
    a.n_pages = n_pages;
    a.free_pages = free_pages;
    a.pool = pool;
    a.pool_out = pool_out;
    a.table = const_cast<int32_t*>(table);
    a.stride = table_stride;
    a.err = err_dev;
    return run_plan<true>(a, (cudaStream_t)stream);
}

extern "C" int llama_paged_store(const void* k, const void* v, int batch, int tokens, int src_seq, int src_pos,
                                 const int32_t* slots, int n_kv_heads, int head_dim, int dtype,
                                 const llama_paged_cache* kv, int32_t* err_dev, void* stream) {
    if (batch < 0 || tokens < 0 || src_pos < 0 || batch > 65535) return LLAMA_ERR_INVALID_ARG;
    const int rc = paged_cache_check(kv, n_kv_heads, head_dim, dtype);
    if (rc != LLAMA_OK) return rc;
    if ((long long)src_pos + tokens > src_seq) return LLAMA_ERR_POS_RANGE;
    if (batch == 0 || tokens == 0) return LLAMA_OK;
    if (!k || !v || !slots || !aligned16(k) || !aligned16(v)) return LLAMA_ERR_INVALID_ARG;
    StoreArgs a{};
    a.k = (const uint4*)k;
    a.v = (const uint4*)v;
    a.pk = (uint4*)kv->k;
    a.pv = (uint4*)kv->v;
    a.slots = slots;
    a.tokens = tokens;
    a.src_seq = src_seq;
    a.src_pos = src_pos;
    a.n_kv_heads = n_kv_heads;
    a.shift = page_shift(kv->page_size);
    a.log_vec = row_log_vec(head_dim, dtype);
    a.n_slots = (long long)kv->n_pages * kv->page_size;
    a.err = err_dev;
    const long long vecs = (long long)tokens << a.log_vec;
    const dim3 grid((unsigned)((vecs + kStoreThreads * kStoreVec - 1) / (kStoreThreads * kStoreVec)), n_kv_heads, batch);
    return launch_pdl(k_paged_store, grid, dim3(kStoreThreads), 0, (cudaStream_t)stream, a) == cudaSuccess
               ? LLAMA_OK
               : LLAMA_ERR_CUDA;
}

extern "C" int llama_beam_reorder(const int32_t* parents, int groups, int beams, const int32_t* lens, int32_t* table,
                                  int table_stride, const llama_paged_cache* caches, int n_layers, int n_kv_heads,
                                  int head_dim, int dtype, int32_t* err_dev, void* stream) {
    if (groups < 0 || groups > 65535 || beams < 1 || n_layers < 1 || n_layers > kReorderLayers || table_stride <= 0)
        return LLAMA_ERR_INVALID_ARG;
    if (beams > kMaxBeams) return LLAMA_ERR_UNSUPPORTED_DIMS;
    if (!caches) return LLAMA_ERR_INVALID_ARG;
    ReorderArgs a{};
    for (int l = 0; l < n_layers; ++l) {
        const int rc = paged_cache_check(&caches[l], n_kv_heads, head_dim, dtype);
        if (rc != LLAMA_OK) return rc;
        if (caches[l].n_pages != caches[0].n_pages || caches[l].page_size != caches[0].page_size)
            return LLAMA_ERR_INVALID_ARG;   // one table addresses every layer
        a.kv[2 * l] = (uint4*)caches[l].k;
        a.kv[2 * l + 1] = (uint4*)caches[l].v;
    }
    if (groups == 0 || beams == 1) return LLAMA_OK;   // a beam alone keeps its state
    if (!parents || !lens || !table) return LLAMA_ERR_INVALID_ARG;
    a.parents = parents;
    a.lens = lens;
    a.table = table;
    a.beams = beams;
    a.stride = table_stride;
    a.shift = page_shift(caches[0].page_size);
    a.n_pages = caches[0].n_pages;
    a.n_kv_heads = n_kv_heads;
    a.log_vec = row_log_vec(head_dim, dtype);
    a.n_layers = n_layers;
    a.err = err_dev;
    const long long most = ((long long)n_kv_heads * (caches[0].page_size - 1)) << a.log_vec;   // vectors of one page
    const long long want = (most + kReorderThreads - 1) / kReorderThreads;
    const dim3 grid((unsigned)std::min<long long>(std::max<long long>(want, 1), 64), 2 * n_layers + 1, groups);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (beams <= 4) e = launch_pdl(k_beam_reorder<4>, grid, dim3(kReorderThreads), 0, s, a);
    else if (beams <= 8) e = launch_pdl(k_beam_reorder<8>, grid, dim3(kReorderThreads), 0, s, a);
    else if (beams <= 16) e = launch_pdl(k_beam_reorder<16>, grid, dim3(kReorderThreads), 0, s, a);
    else e = launch_pdl(k_beam_reorder<32>, grid, dim3(kReorderThreads), 0, s, a);
    return e == cudaSuccess ? LLAMA_OK : LLAMA_ERR_CUDA;
}
