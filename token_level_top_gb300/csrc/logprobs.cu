// logprobs.cu -- log probabilities of given tokens, entropy and the most likely
// alternatives, read off a row of logits, and their gradient.
//
// Forward: one block per row; the row's maximum, then the sums, then n_top
// rounds that each take the best entry after the one before.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <class T>
__device__ __forceinline__ float value(const T* p, long long i)
{
    return static_cast<float>(p[i]);
}

// Orders (value, index) pairs: larger value first, then lower index; NaN last.
__device__ __forceinline__ uint64_t rank_key(float x, int i)
{
    uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
    b = b & 0x80000000u ? ~b : b | 0x80000000u;
    if (x != x) b = 0;
    return (static_cast<uint64_t>(b) << 32) | static_cast<uint32_t>(~i);
}

__device__ float block_sum(float x, float* s)
{
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.0f;
    for (int i = 0; i < kThreads / 32; ++i) x += s[i];
    __syncthreads();
    return x;
}

template <class T>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const LogprobArgs a)
{
    __shared__ float s_f[kThreads / 32];
    __shared__ uint64_t s_k[kThreads / 32];
    const long long row = blockIdx.x;
    const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
    float m = -INFINITY;
    bool nan = false;
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) {
        const float v = value(x, i);
        nan |= v != v;
        m = fmaxf(m, v);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if ((threadIdx.x & 31) == 0) s_f[threadIdx.x >> 5] = m;
    nan = __syncthreads_or(nan);
    for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, s_f[i]);
    __syncthreads();
    if (nan && threadIdx.x == 0) record_error(a.status, MOE_ERR_NONFINITE);
    const float ref = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, w = 0.0f;
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) {
        const float z = value(x, i) - ref, e = expf(z);
        l += e;
        if (e != 0.0f) w += e * z;
    }
    l = block_sum(l, s_f);
    w = block_sum(w, s_f);
    const bool none = m == -INFINITY && !nan;
    const float log_l = logf(l);
    const float lse = ref + log_l;
    if (threadIdx.x == 0) {
        if (a.lse) a.lse[row] = lse;
        if (a.entropy) a.entropy[row] = none ? 0.0f : log_l - w / l;
        if (a.logprob) {
            const int t = a.token[row];
            float lp = 0.0f;
            if (t >= a.vocab) record_error(a.status, MOE_ERR_INDEX);
            if (t >= 0 && t < a.vocab) {
                const float v = value(x, t);
                lp = none ? -INFINITY : v - ref - log_l;
            }
            a.logprob[row] = lp;
        }
    }
    uint64_t last = ~0ull;
    for (int n = 0; n < a.n_top; ++n) {
        uint64_t best = 0;
        for (int i = threadIdx.x; i < a.vocab; i += kThreads) {
            const uint64_t k = rank_key(value(x, i), i);
            if (k < last && k > best) best = k;
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            const uint64_t o = __shfl_xor_sync(0xffffffffu, best, off);
            best = o > best ? o : best;
        }
        if ((threadIdx.x & 31) == 0) s_k[threadIdx.x >> 5] = best;
        __syncthreads();
        for (int i = 0; i < kThreads / 32; ++i) best = s_k[i] > best ? s_k[i] : best;
        __syncthreads();
        if (threadIdx.x == 0) {
            const int id = best ? static_cast<int>(~static_cast<uint32_t>(best)) : -1;
            a.top_ids[row * a.n_top + n] = id;
            a.top_logprobs[row * a.n_top + n] = id < 0 || none ? -INFINITY : value(x, id) - ref - log_l;
        }
        last = best;
    }
}

// dx_i = g (1[i = token] - p_i) - h p_i (ln p_i + H).
template <class T>
__global__ void __launch_bounds__(kThreads) token_logprobs_backward_kernel(const LogprobGradArgs a)
{
    const long long row = blockIdx.x;
    const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
    T* dx = static_cast<T*>(a.dlogits) + row * a.drow_stride;
    int t = a.token ? a.token[row] : -1;
    if (t >= a.vocab) {
        if (threadIdx.x == 0) record_error(a.status, MOE_ERR_INDEX);
        t = -1;
    }
    const float lse = a.lse[row], H = a.entropy ? a.entropy[row] : 0.0f;
    const float g = t >= 0 && a.dlogprob ? a.dlogprob[row] : 0.0f, h = a.dentropy ? a.dentropy[row] : 0.0f;
    const bool none = lse == -INFINITY;   // nothing live in the row: no probability to move
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) {
        const float z = value(x, i) - lse, p = none ? 0.0f : expf(z);
        float d = -g * p;
        if (p != 0.0f) d -= h * p * (z + H);
        if (i == t && !none) d += g;
        dx[i] = static_cast<T>(d);
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t s)
{
    if (a.rows <= 0) return cudaSuccess;
    const unsigned grid = static_cast<unsigned>(a.rows);
    if (a.bf16)
        token_logprobs_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
    else
        token_logprobs_kernel<float><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_token_logprobs_backward(const LogprobGradArgs& a, cudaStream_t s)
{
    if (a.rows <= 0) return cudaSuccess;
    const unsigned grid = static_cast<unsigned>(a.rows);
    if (a.bf16)
        token_logprobs_backward_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
    else
        token_logprobs_backward_kernel<float><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
