// attention.cu -- attention of one new token per sequence over the paged cache.
//
// One block per (query head, sequence): each warp takes every eighth live key,
// its lanes hold D/32 dimensions each, and keeps the running maximum and sum of
// its softmax; the eight partial results are joined in shared memory.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;

template <int D, bool kE4m3>
__global__ void __launch_bounds__(32 * kWarps) paged_attention_kernel(const AttentionArgs a)
{
    constexpr int kPer = D / 32;
    __shared__ float s_m[kWarps], s_l[kWarps];
    __shared__ float s_o[kWarps][D];
    const int h = blockIdx.x, b = blockIdx.y;
    const int hk = h / (a.n_heads / a.n_kv_heads);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const long long most = static_cast<long long>(a.max_pages) * a.page_size;
    long long n = a.seq_len[b];
    if (n < 0 || n > most) {
        if (threadIdx.x == 0) record_error(a.status, MOE_ERR_INDEX);
        n = n < 0 ? 0 : most;
    }
    const int len = static_cast<int>(n);
    const int first = a.window > 0 && len > a.window ? len - a.window : 0;
    const __nv_bfloat16* q = a.q + b * a.q_token_stride + h * a.q_head_stride + lane * kPer;
    float qf[kPer], o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        qf[i] = __bfloat162float(q[i]) * a.scale;
        o[i] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int j = first + w; j < len; j += kWarps) {
        const int page = a.page_table[b * a.table_stride + j / a.page_size];
        if (page < 0 || page >= a.n_pages) {
            if (lane == 0) record_error(a.status, MOE_ERR_INDEX);
            continue;
        }
        const long long row = page * a.page_stride + (j % a.page_size) * a.token_stride + hk * a.head_stride + lane * kPer;
        float kf[kPer], vf[kPer], ks = 1.0f, vs = 1.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (kE4m3) {
                kf[i] = float(static_cast<const __nv_fp8_e4m3*>(a.k)[row + i]);
                vf[i] = float(static_cast<const __nv_fp8_e4m3*>(a.v)[row + i]);
            } else {
                kf[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.k)[row + i]);
                vf[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.v)[row + i]);
            }
        }
        if (kE4m3) {
            const long long e = page * a.exp_page_stride + (j % a.page_size) * a.exp_token_stride + hk * a.exp_head_stride;
            ks = exp2f(static_cast<float>(a.k_exp[e]) - 127.0f);
            vs = exp2f(static_cast<float>(a.v_exp[e]) - 127.0f);
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) s += qf[i] * kf[i];
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= ks;
        const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.0f : mn;
        const float f = expf(m - ref), p = expf(s - ref);
        l = l * f + p;
        m = mn;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + p * vs * vf[i];
    }
    if (lane == 0) {
        s_m[w] = m;
        s_l[w] = l;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) s_o[w][lane * kPer + i] = o[i];
    __syncthreads();
    float M = -INFINITY;
    for (int i = 0; i < kWarps; ++i) M = fmaxf(M, s_m[i]);
    const float ref = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    for (int i = 0; i < kWarps; ++i) L += s_l[i] * expf(s_m[i] - ref);
    const bool empty = L == 0.0f;
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float x = 0.0f;
        for (int i = 0; i < kWarps; ++i) x += s_o[i][d] * expf(s_m[i] - ref);
        a.out[b * a.out_token_stride + h * a.out_head_stride + d] = __float2bfloat16(empty ? 0.0f : x / L);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[static_cast<long long>(b) * a.n_heads + h] = empty ? -INFINITY : ref + logf(L);
}

}  // namespace

size_t paged_attention_ws_bytes(int head_dim)
{
    return head_dim == 64 || head_dim == 128 || head_dim == 256 ? 256 : 0;
}

template <int D>
static cudaError_t launch_d(const AttentionArgs& a, bool e4m3, cudaStream_t s)
{
    const dim3 grid(a.n_heads, a.B);
    if (e4m3)
        paged_attention_kernel<D, true><<<grid, 32 * kWarps, 0, s>>>(a);
    else
        paged_attention_kernel<D, false><<<grid, 32 * kWarps, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_attention(const AttentionArgs& a, int head_dim, bool e4m3, cudaStream_t s)
{
    if (a.B <= 0) return cudaSuccess;
    switch (head_dim) {
        case 64: return launch_d<64>(a, e4m3, s);
        case 128: return launch_d<128>(a, e4m3, s);
        default: return launch_d<256>(a, e4m3, s);
    }
}

}  // namespace moe
