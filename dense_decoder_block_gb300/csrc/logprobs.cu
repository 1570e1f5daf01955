// llama_token_logprobs: log probabilities of given tokens, entropy and top alternatives of fp32 logits.
//
// With m = max z = z_u (u the first such token) and e_v = e^(z_v - m), d = sum_{v != u} e_v and
// t = sum e_v (z_v - m) (terms of weight 0 left out):
//   log p_v = (z_v - m) - log(1 + d),   H = log(1 + d) - t / (1 + d),
// all without cancellation: the terms of t are <= 0, and leaving the 1 out of the sums keeps small d.
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace llama {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTop = 32;

struct LogprobArgs {
    const float* logits;
    int rows, vocab, n_top;
    const int* tokens;
    float* logprobs;
    float* entropy;
    int* top_ids;
    float* top_logprobs;
    int* err;
};

// Larger logits first, equal ones by increasing token; a NaN counts as the lowest value, so that every order is total.
__device__ __forceinline__ unsigned long long order_key(float z, int v) {
    if (!(z == z)) z = -INFINITY;
    if (z == 0.f) z = 0.f;   // -0 and 0 are equal
    const unsigned u = __float_as_uint(z);
    const unsigned o = u & 0x80000000u ? ~u : u | 0x80000000u;
    return (unsigned long long)o << 32 | (0xffffffffu - (unsigned)v);
}

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T x, T* s, F&& f) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = f(x, __shfl_xor_sync(0xffffffffu, x, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    x = s[0];
    for (int w = 1; w < kThreads / 32; ++w) x = f(x, s[w]);
    return x;
}

__global__ void __launch_bounds__(kThreads) k_logprobs(const LogprobArgs a) {
    __shared__ unsigned long long s_key[kThreads / 32];
    __shared__ double s_sum[kThreads / 32];
    ptx::griddep_wait();
    const int r = blockIdx.x, V = a.vocab;
    int token = 0;
    if (a.tokens) {
        token = a.tokens[r];
        if (token < 0 || token >= V) {
            if (token >= V && threadIdx.x == 0) record_error(a.err, LLAMA_ERR_INVALID_ARG);
            return;
        }
    }
    const float* z = a.logits + (size_t)r * V;
    unsigned long long first = 0;
    float nan = 0.f;
    for (int v = threadIdx.x; v < V; v += kThreads) {
        const float x = z[v];
        first = max(first, order_key(x, v));
        if (!(x < INFINITY)) nan = NAN;   // NaN or +inf
    }
    first = block_reduce<unsigned long long>(first, s_key, [](auto x, auto y) { return x > y ? x : y; });
    const double bad = block_reduce<double>(nan, s_sum, [](double x, double y) { return x + y; });
    const int u = (int)(0xffffffffu - (unsigned)first);
    const float m = z[u];
    const bool empty = m == -INFINITY && bad == 0.0;
    double s = 0.0, t = 0.0;
    if (!empty) {
        float fs = 0.f, ft = 0.f;
        for (int v = threadIdx.x; v < V; v += kThreads) {
            const float x = z[v] - m, e = expf(x);
            if (v != u) fs += e;
            if (e > 0.f) ft = fmaf(e, x, ft);
        }
        s = fs;
        t = ft;
    }
    s = block_reduce<double>(s, s_sum, [](double x, double y) { return x + y; }) + bad;
    t = block_reduce<double>(t, s_sum, [](double x, double y) { return x + y; });
    const double lse = log1p(s);
    auto logprob = [&](float x) { return empty ? -INFINITY : (float)((double)(x - m) - lse); };
    if (threadIdx.x == 0) {
        if (a.tokens) a.logprobs[r] = logprob(z[token]);
        if (a.entropy) a.entropy[r] = empty ? 0.f : (float)(lse - t / (1.0 + s));
    }
    unsigned long long above = ~0ull;
    for (int k = 0; k < a.n_top; ++k) {
        unsigned long long best = 0;
        for (int v = threadIdx.x; v < V; v += kThreads) {
            const unsigned long long key = order_key(z[v], v);
            if (key < above && key > best) best = key;
        }
        best = block_reduce<unsigned long long>(best, s_key, [](auto x, auto y) { return x > y ? x : y; });
        above = best;
        if (threadIdx.x == 0) {
            const int v = (int)(0xffffffffu - (unsigned)best);
            a.top_ids[(size_t)r * a.n_top + k] = v;
            a.top_logprobs[(size_t)r * a.n_top + k] = logprob(z[v]);
        }
    }
}

}  // namespace
}  // namespace llama

using namespace llama;

extern "C" int llama_token_logprobs(const float* logits, int rows, int vocab, const int32_t* tokens, int n_top,
                                    float* logprobs, float* entropy, int32_t* top_ids, float* top_logprobs,
                                    int32_t* err_dev, void* stream) {
    if (rows < 0 || vocab <= 0 || vocab > (1 << 20) || n_top < 0 || n_top > kMaxTop || n_top > vocab)
        return LLAMA_ERR_INVALID_ARG;
    if ((tokens == nullptr) != (logprobs == nullptr)) return LLAMA_ERR_INVALID_ARG;
    if (rows == 0) return LLAMA_OK;
    if (!logits || (n_top > 0 && (!top_ids || !top_logprobs))) return LLAMA_ERR_INVALID_ARG;
    LogprobArgs a{logits, rows, vocab, n_top, tokens, logprobs, entropy, top_ids, top_logprobs, err_dev};
    return launch_pdl(k_logprobs, dim3(rows), dim3(kThreads), 0, (cudaStream_t)stream, a) == cudaSuccess ? LLAMA_OK
                                                                                                       : LLAMA_ERR_CUDA;
}
