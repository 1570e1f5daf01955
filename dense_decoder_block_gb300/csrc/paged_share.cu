// Pages that rows of a block table share: forking a row (its full pages shared, its unfilled one
// copied) and giving rows up (pages without a holder go back on the stack).
//
// refs[p] counts the holders of page p beside the first, so a page as llama_paged_plan hands it out
// has the count 0 and the calls that know nothing of sharing need not touch it.
//
// As in paged.cu, kernels are launched with programmatic stream serialization, wait for the kernels
// before them before they read anything, and let their dependents start only when they end.
#include <algorithm>
#include <climits>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int kShareThreads = 1024;
constexpr int kMaxRows = 65536;                // rows of a table: one bit each in shared memory
constexpr int kRowWords = kMaxRows / 32;

// Sets the row's bit; true when it was set before.
__device__ __forceinline__ bool mark(unsigned* bits, int row) {
    const unsigned m = 1u << (row & 31);
    return atomicOr(bits + (row >> 5), m) & m;
}
__device__ __forceinline__ bool marked(const unsigned* bits, int row) { return bits[row >> 5] >> (row & 31) & 1; }

// Exclusive prefix of x over the 1024 threads of the CTA, and the total.  s: 32 words.
__device__ __forceinline__ int block_prefix(int x, int* s, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += v;
    }
    __syncthreads();   // s may still be read from a previous use
    if (lane == 31) s[warp] = y;
    __syncthreads();
    int w = s[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += v;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return y - x + (warp ? before : 0);
}

// ----------------------------------------------------------------------------- fork
// Two launches: one CTA checks the forks against one another, takes the fresh pages and leaves a job
// for each fork; a grid over (layer and K or V, fork) then copies rows, table entries and counts.
struct ForkArgs {
    const int* src;
    const int* dst;
    const int* lens;
    int n;
    int* refs;
    const int* free_pages;
    const int* pool;
    int* pool_out;
    int* table;
    int rows, stride, shift, n_pages, n_kv_heads, log_vec, n_layers;
    int4* jobs;   // {source row, row, full pages, rows of the unfilled one}
    int* err;
};
constexpr int kForkLayers = 128;
struct ForkCaches {
    uint4* kv[2 * kForkLayers];   // K and V of each layer
};

__global__ void __launch_bounds__(kShareThreads) k_fork_jobs(const ForkArgs a) {
    __shared__ unsigned s_once[kRowWords], s_twice[kRowWords], s_source[kRowWords];
    __shared__ int s_scan[32];
    const int tid = threadIdx.x;
    ptx::griddep_wait();
    const int n_free = __ldcg(a.pool);
    // the first forks, one a thread, are read once (each read is a round trip of the call)
    int3 mine = make_int3(-1, -1, -1);
    if (tid < a.n) mine = make_int3(__ldcg(a.src + tid), __ldcg(a.dst + tid), __ldcg(a.lens + tid));
    auto words = [&](int i) { return i == tid ? mine : make_int3(__ldcg(a.src + i), __ldcg(a.dst + i), __ldcg(a.lens + i)); };
    for (int i = tid; i < (a.rows + 31) >> 5; i += kShareThreads) s_once[i] = s_twice[i] = s_source[i] = 0;
    __syncthreads();
    for (int i = tid; i < a.n; i += kShareThreads) {
        const int3 w = words(i);
        if (w.y >= 0 && w.y < a.rows && mark(s_once, w.y)) mark(s_twice, w.y);
        if (w.x >= 0 && w.x < a.rows) mark(s_source, w.x);
    }
    __syncthreads();
    // a fork's full pages and unfilled rows; none of either when it is left out
    auto fork = [&](int i, bool record) -> int4 {
        const int3 w = words(i);
        int4 j = make_int4(w.x, w.y, 0, 0);
        const int len = w.z;
        if (j.x < 0 || j.x >= a.rows || j.y < 0 || j.y >= a.rows || marked(s_twice, j.y) || marked(s_source, j.y)) {
            if (record) record_error(a.err, LLAMA_ERR_INVALID_ARG);
        } else if (len < 0 || len > (long long)a.stride << a.shift) {
            if (record) record_error(a.err, LLAMA_ERR_POS_RANGE);
        } else {
            j.z = len >> a.shift;
            j.w = len & ((1 << a.shift) - 1);
        }
        return j;
    };
    int total = 0;
    for (int i0 = 0; i0 < a.n; i0 += kShareThreads) {
        const int i = i0 + tid;
        total += __syncthreads_count(i < a.n && fork(i, true).w > 0);
    }
    const bool pool_ok = n_free >= 0 && n_free <= a.n_pages;
    const bool enough = pool_ok && total <= n_free;
    if (!enough && tid == 0) record_error(a.err, pool_ok ? LLAMA_ERR_NO_PAGES : LLAMA_ERR_INVALID_ARG);
    int done = 0;
    for (int i0 = 0; i0 < a.n; i0 += kShareThreads) {
        const int i = i0 + tid;
        int4 j = make_int4(0, 0, 0, 0);
        if (i < a.n && enough) j = fork(i, false);
        int here;
        const int o = done + block_prefix(j.w > 0, s_scan, here);
        done += here;
        if (j.w > 0) {
            const int id = __ldcg(a.free_pages + (n_free - 1 - o));
            if (id < 0 || id >= a.n_pages) record_error(a.err, LLAMA_ERR_INVALID_ARG);
            a.table[(size_t)j.y * a.stride + j.z] = id;
        }
        if (i < a.n) a.jobs[i] = j;
    }
    if (tid == 0) {
        a.pool_out[0] = n_free - (enough ? total : 0);
        a.pool_out[1] = 0;
    }
}

// The copies of a fork -- the rows of one head, in K and V of every layer -- are one list, cut over the warps of
// gridDim.y - 1 CTAs; a lane has kCopyVec loads under way.  (A CTA per layer and K or V read jobs and tables again and was
// mostly waiting: 112 forks of 32 layers 37 us.  A list of single vectors took a division for each: 30 us, so 23.5, at 0.86
// of the copy rate.)  The last CTA of a fork moves its table entries.
constexpr int kCopyThreads = 256;
constexpr int kCopyVec = 8;
constexpr int kCopyCtas = 16;   // per SM: from here on a CTA takes more

__global__ void __launch_bounds__(kCopyThreads) k_fork_copy(const ForkArgs a, const __grid_constant__ ForkCaches c) {
    ptx::griddep_wait();
    const int4 j = __ldcg(a.jobs + blockIdx.x);
    const int* from = a.table + (size_t)j.x * a.stride;
    int* to = a.table + (size_t)j.y * a.stride;
    const int parts = gridDim.y - 1;
    if ((int)blockIdx.y == parts) {   // table entries and counts
        for (int e = threadIdx.x; e < j.z; e += kCopyThreads) {
            const int id = __ldcg(from + e);
            to[e] = id;
            if (id >= 0 && id < a.n_pages) atomicAdd(a.refs + id, 1);
            else record_error(a.err, LLAMA_ERR_INVALID_ARG);
        }
        return;
    }
    if (j.w == 0) return;
    const int sp = __ldcg(from + j.z), dp = __ldcg(to + j.z);
    if (dp < 0 || dp >= a.n_pages) return;   // recorded when it was taken
    if (sp < 0 || sp >= a.n_pages) {
        if (blockIdx.y == 0 && threadIdx.x == 0) record_error(a.err, LLAMA_ERR_INVALID_ARG);
        return;
    }
    const size_t page = (size_t)a.n_kv_heads << (a.shift + a.log_vec);
    const int run = j.w << a.log_vec, lane = threadIdx.x & 31;   // vectors of a head
    const int heads = 2 * a.n_layers * a.n_kv_heads, step = parts * (kCopyThreads / 32);
    for (int u = blockIdx.y * (kCopyThreads / 32) + (threadIdx.x >> 5); u < heads; u += step) {
        const int b = u / a.n_kv_heads;
        const size_t at = (size_t)(u - b * a.n_kv_heads) << (a.shift + a.log_vec);
        const uint4* src = c.kv[b] + sp * page + at;
        uint4* dst = c.kv[b] + dp * page + at;
        for (int x0 = lane; x0 < run; x0 += 32 * kCopyVec) {
            uint4 v[kCopyVec];
#pragma unroll
            for (int i = 0; i < kCopyVec; ++i)
                if (x0 + 32 * i < run) v[i] = __ldcg(src + x0 + 32 * i);
#pragma unroll
            for (int i = 0; i < kCopyVec; ++i)
                if (x0 + 32 * i < run) dst[x0 + 32 * i] = v[i];
        }
    }
}

// ----------------------------------------------------------------------------- free
// Entries (row i of the call, page j of the row) are numbered in order, e = prefix[i] + j.  An entry
// gives up one hold on its page; the last entry of a page (the largest e) settles it: with d entries
// of the page and h = refs + 1 holders, d < h leaves refs - d, d >= h sends the page back.  The k-th
// page of F that goes back lies at n_free + F - 1 - k of the stack.
//
// One cluster (one CTA where there are few entries), its warps with runs of entries of one length,
// and barriers of the cluster between the steps: clear the pages' words, count and take the maximum
// (atomics whose order does not matter), count what goes back per warp, write.  A thread keeps its first
// entries' pages and outcomes in registers.  The pages' words lie in the workspace and are cleared for the
// pages of the call alone, so the cost does not grow with the cache.  Bound by round trips and the barriers: 189 entries of 3
// rows 5 us, 4536 of 112 rows 11.
struct FreeArgs {
    const int* list;
    const int* lens;
    int n, rows, stride, shift, n_pages;
    int* refs;
    int* free_pages;
    const int* pool;
    int* pool_out;
    const int* table;
    int* drops;     // [n_pages]
    int* last;      // [n_pages]
    int* prefix;    // [n + 1]; calls of few rows keep it in shared memory
    int* counts;    // [kFreeCtas * 32]: pages that go back, per warp
    int* err;
};
constexpr int kFreeCtas = 8;
constexpr int kFewRows = 2048;
constexpr int kKept = 4;        // entries of a thread in registers

__global__ void __launch_bounds__(kShareThreads) k_paged_free(const FreeArgs a) {
    __shared__ unsigned s_once[kRowWords], s_twice[kRowWords];
    __shared__ int s_prefix[kFewRows + 1], s_row[kFewRows];
    __shared__ int s_scan[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = gridDim.x;   // one cluster
    ptx::griddep_wait();
    const int n_free = __ldcg(a.pool);
    const bool pool_ok = n_free >= 0 && n_free <= a.n_pages;
    if (a.n == 0) {   // one CTA, no workspace
        if (tid == 0) {
            if (!pool_ok) record_error(a.err, LLAMA_ERR_INVALID_ARG);
            a.pool_out[0] = n_free;
            a.pool_out[1] = 0;
        }
        return;
    }
    auto sync = [&] {
        if (ctas > 1) ptx::cluster_sync();
        else __syncthreads();
    };
    // Where each row's entries begin: of few rows every CTA finds out by itself, of many the first does.
    const bool few = a.n <= kFewRows;
    if (few || blockIdx.x == 0) {
        const int2 mine = tid < a.n ? make_int2(__ldcg(a.list + tid), __ldcg(a.lens + tid)) : make_int2(-1, -1);
        for (int i = tid; i < (a.rows + 31) >> 5; i += kShareThreads) s_once[i] = s_twice[i] = 0;
        __syncthreads();
        for (int i = tid; i < a.n; i += kShareThreads) {
            const int r = i == tid ? mine.x : __ldcg(a.list + i);
            if (r >= 0 && r < a.rows && mark(s_once, r)) mark(s_twice, r);
        }
        __syncthreads();
        int run = 0;
        for (int i0 = 0; i0 < a.n; i0 += kShareThreads) {
            const int i = i0 + tid;
            int pages = 0;
            if (i < a.n) {
                const int r = i0 == 0 ? mine.x : __ldcg(a.list + i), len = i0 == 0 ? mine.y : __ldcg(a.lens + i);
                int bad = 0;
                if (r < 0 || r >= a.rows || marked(s_twice, r)) bad = LLAMA_ERR_INVALID_ARG;
                else if (len < 0 || len > (long long)a.stride << a.shift) bad = LLAMA_ERR_POS_RANGE;
                else pages = (int)(((long long)len + (1 << a.shift) - 1) >> a.shift);
                if (bad && blockIdx.x == 0) record_error(a.err, bad);
                if (few) s_row[i] = r;
            }
            int here;
            const int before = block_prefix(pages, s_scan, here);
            if (i < a.n) (few ? s_prefix : a.prefix)[i] = run + before;
            run += here;
        }
        if (tid == 0) (few ? s_prefix : a.prefix)[a.n] = run;
    }
    if (few) __syncthreads();
    else sync();
    auto prefix = [&](int i) { return few ? s_prefix[i] : __ldcg(a.prefix + i); };
    const int total = prefix(a.n);
    const int wid = blockIdx.x * 32 + warp, warps = ctas * 32;
    const int e0 = (int)((long long)total * wid / warps), e1 = (int)((long long)total * (wid + 1) / warps);
    auto page_at = [&](int e) -> int {   // of entry e, -2 when it is no page
        int lo = 0;   // the last row whose entries start at or before e
        for (int hi = a.n - 1; lo < hi;) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix(mid) <= e) lo = mid;
            else hi = mid - 1;
        }
        const int id = __ldcg(a.table + (size_t)(few ? s_row[lo] : __ldcg(a.list + lo)) * a.stride + (e - prefix(lo)));
        return id < 0 || id >= a.n_pages ? -2 : id;
    };
    int page[kKept];   // -1: no entry
#pragma unroll
    for (int k = 0; k < kKept; ++k) page[k] = e0 + 32 * k + lane < e1 ? page_at(e0 + 32 * k + lane) : -1;
    // f(place among this thread's entries, entry, page) for this warp's entries, 32 at a time
    auto entries = [&](auto&& f) {
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            if (e0 + 32 * k < e1) f(k, e0 + 32 * k + lane, page[k]);
        for (int e = e0 + 32 * kKept + lane; e - lane < e1; e += 32) f(kKept, e, e < e1 ? page_at(e) : -1);
    };
    entries([&](int, int, int id) {
        if (id == -2) record_error(a.err, LLAMA_ERR_INVALID_ARG);
        if (id >= 0) {
            a.drops[id] = 0;
            a.last[id] = -1;
        }
    });
    sync();
    entries([&](int, int e, int id) {
        if (id >= 0) {
            atomicAdd(a.drops + id, 1);
            atomicMax(a.last + id, e);
        }
    });
    sync();
    // Of the entry that settles its page: the holds left (below 0: given up more often than held); kOther: another does.
    constexpr int kOther = INT_MAX;
    auto settle = [&](int e, int id) -> int {
        if (id < 0) return kOther;
        const int last = __ldcg(a.last + id), drops = __ldcg(a.drops + id), refs = __ldcg(a.refs + id);
        return last == e ? max(refs, 0) + 1 - drops : kOther;
    };
    int left[kKept];
    int mine = 0;
    entries([&](int k, int e, int id) {
        const int x = settle(e, id);
        if (k < kKept) left[k] = x;
        mine += __popc(__ballot_sync(0xffffffffu, x <= 0));
    });
    if (lane == 0) a.counts[wid] = mine;
    sync();
    int before = 0, back = 0;
    for (int w = lane; w < warps; w += 32) {
        const int c = __ldcg(a.counts + w);
        back += c;
        before += w < wid ? c : 0;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    back = __reduce_add_sync(0xffffffffu, back);
    const bool room = pool_ok && back <= a.n_pages - n_free;
    if (wid == 0 && lane == 0) {
        if (!room) record_error(a.err, pool_ok ? LLAMA_ERR_NO_PAGES : LLAMA_ERR_INVALID_ARG);
        a.pool_out[0] = n_free + (room ? back : 0);
        a.pool_out[1] = 0;
    }
    if (!room) return;
    entries([&](int k, int e, int id) {
        const int x = k < kKept ? left[k] : settle(e, id);
        const unsigned ones = __ballot_sync(0xffffffffu, x <= 0);
        if (x != kOther) {
            if (x < 0) record_error(a.err, LLAMA_ERR_INVALID_ARG);
            a.refs[id] = max(x - 1, 0);
            if (x <= 0) a.free_pages[n_free + back - 1 - (before + __popc(ones & ((1u << lane) - 1)))] = id;
        }
        before += __popc(ones);
    });
}

}  // namespace
}  // namespace llama

using namespace llama;

extern "C" size_t llama_paged_fork_workspace_bytes(int n) { return n > 0 ? (size_t)n * sizeof(int4) : 0; }

extern "C" int llama_paged_fork(const int32_t* src, const int32_t* dst, const int32_t* lens, int n, int32_t* refs,
                                const int32_t* free_pages, const int32_t* pool, int32_t* pool_out, int32_t* table,
                                int table_rows, int table_stride, const llama_paged_cache* caches, int n_layers,
                                int n_kv_heads, int head_dim, int dtype, void* ws, size_t ws_bytes, int32_t* err_dev,
                                void* stream) {
    if (n < 0 || n > 65535 || n_layers < 1 || n_layers > kForkLayers || table_rows <= 0 || table_stride <= 0)
        return LLAMA_ERR_INVALID_ARG;
    if (table_rows > kMaxRows) return LLAMA_ERR_UNSUPPORTED_DIMS;
    if (!caches) return LLAMA_ERR_INVALID_ARG;
    ForkCaches c{};
    for (int l = 0; l < n_layers; ++l) {
        const int rc = paged_cache_check(&caches[l], n_kv_heads, head_dim, dtype);
        if (rc != LLAMA_OK) return rc;
        if (caches[l].n_pages != caches[0].n_pages || caches[l].page_size != caches[0].page_size)
            return LLAMA_ERR_INVALID_ARG;   // one table addresses every layer
        c.kv[2 * l] = (uint4*)caches[l].k;
        c.kv[2 * l + 1] = (uint4*)caches[l].v;
    }
    if (!paged_pools_ok(pool, pool_out)) return LLAMA_ERR_INVALID_ARG;
    if (n > 0 && (!src || !dst || !lens || !refs || !free_pages || !table)) return LLAMA_ERR_INVALID_ARG;
    if (n > 0 && (!ws || ws_bytes < llama_paged_fork_workspace_bytes(n))) return LLAMA_ERR_WORKSPACE;
    if ((uintptr_t)ws & 15) return LLAMA_ERR_INVALID_ARG;
    ForkArgs a{};
    a.src = src;
    a.dst = dst;
    a.lens = lens;
    a.n = n;
    a.refs = refs;
    a.free_pages = free_pages;
    a.pool = pool;
    a.pool_out = pool_out;
    a.table = table;
    a.rows = table_rows;
    a.stride = table_stride;
    a.shift = page_shift(caches[0].page_size);
    a.n_pages = caches[0].n_pages;
    a.n_kv_heads = n_kv_heads;
    a.log_vec = paged_row_log_vec(head_dim, dtype);
    a.n_layers = n_layers;
    a.jobs = (int4*)ws;
    a.err = err_dev;
    cudaStream_t s = (cudaStream_t)stream;
    if (launch_pdl(k_fork_jobs, dim3(1), dim3(kShareThreads), 0, s, a) != cudaSuccess) return LLAMA_ERR_CUDA;
    if (n == 0) return LLAMA_OK;
    const long long want = (2LL * n_layers * n_kv_heads + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    const long long room = std::max(1, kCopyCtas * device_sm_count() / n);
    const dim3 grid(n, (unsigned)std::min(want, room) + 1);
    return launch_pdl(k_fork_copy, grid, dim3(kCopyThreads), 0, s, a, c) == cudaSuccess ? LLAMA_OK : LLAMA_ERR_CUDA;
}

extern "C" size_t llama_paged_free_workspace_bytes(int n, int n_pages) {
    if (n <= 0 || n_pages <= 0) return 0;
    return ((size_t)2 * n_pages + n + 1 + kFreeCtas * 32) * sizeof(int);
}

extern "C" int llama_paged_free(const int32_t* list, const int32_t* lens, int n, int page_size, int n_pages, int32_t* refs,
                                int32_t* free_pages, const int32_t* pool, int32_t* pool_out, const int32_t* table,
                                int table_rows, int table_stride, void* ws, size_t ws_bytes, int32_t* err_dev, void* stream) {
    if (n < 0 || n > kMaxRows || table_rows <= 0 || table_stride <= 0) return LLAMA_ERR_INVALID_ARG;
    const int rc = paged_geometry_check(page_size, n_pages);
    if (rc != LLAMA_OK) return rc;
    if (table_rows > kMaxRows || (long long)n * table_stride > INT32_MAX - 1024) return LLAMA_ERR_UNSUPPORTED_DIMS;
    if (!paged_pools_ok(pool, pool_out)) return LLAMA_ERR_INVALID_ARG;
    if (n > 0 && (!list || !lens || !refs || !free_pages || !table)) return LLAMA_ERR_INVALID_ARG;
    if (n > 0 && (!ws || ws_bytes < llama_paged_free_workspace_bytes(n, n_pages))) return LLAMA_ERR_WORKSPACE;
    if ((uintptr_t)ws & 15) return LLAMA_ERR_INVALID_ARG;
    FreeArgs a{};
    a.list = list;
    a.lens = lens;
    a.n = n;
    a.rows = table_rows;
    a.stride = table_stride;
    a.shift = page_shift(page_size);
    a.n_pages = n_pages;
    a.refs = refs;
    a.free_pages = free_pages;
    a.pool = pool;
    a.pool_out = pool_out;
    a.table = table;
    a.drops = (int*)ws;
    a.last = a.drops + n_pages;
    a.prefix = a.last + n_pages;
    a.counts = a.prefix + n + 1;
    a.err = err_dev;
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = (long long)n * table_stride <= kShareThreads
                              ? launch_pdl(k_paged_free, dim3(1), dim3(kShareThreads), 0, s, a)
                              : launch_pdl_cluster(k_paged_free, dim3(kFreeCtas), dim3(kShareThreads), 0, kFreeCtas, s, a);
    return e == cudaSuccess ? LLAMA_OK : LLAMA_ERR_CUDA;
}
