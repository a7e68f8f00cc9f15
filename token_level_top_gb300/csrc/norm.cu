// norm.cu -- the root-mean-square norm of rows, with a residual's addition before
// it and an e4m3 output with a scale per row behind it, and its gradient.
//
//   s = x + residual (rounded to the rows' type), r = (mean s^2 + eps)^(-1/2),
//   y = s r w,  scale = max|y| / 448,  code = e4m3(y / scale)
//   dx = r (w dy - u mean(w dy u)) + dsum,  dw = sum over rows of dy u,  u = s r
//
// All of it is memory traffic: a row is read once into registers and everything
// is computed from there.  W warps share a row (1 to 32), each lane P pieces of it;
// a piece is 16 bytes, or one value where a row does not start on 16 bytes.  The
// forward takes a block per row (or several short rows); the gradient keeps its
// blocks over many rows, since a thread sums dw of its columns in registers; the
// blocks' sums go to the workspace and a second kernel adds them in a fixed order.
// r is computed again from s in the gradient: s is read anyway.
//
// Measured on rows in memory (the copy rate is 6.7 TB/s): 16384 x 4096 bf16 with a
// residual 79 us, at the copy rate; its gradient with fp32 dy 113 us, 0.89 of it, the
// weights' sum being 5 us of that.  64 rows: 4 us, a launch and one chain of loads.  Rows
// of 1407 fp32 are taken value by value: the gradient of 5001 21.6 us, 0.58.  The gradient of
// 67 million bf16 values (fp32 dy, dsum) in rows of 512 / 1000 / 2048 / 5120 / 8192 / 16384:
// 0.86 / 0.74 / 0.79 / 0.56 / 0.71 / 0.80 of the copy rate; of 33 million fp32 ones in rows of
// 512 to 4096 0.9, of 8192 0.83.
//
// Squares are summed in fp32.  A row whose sum is not finite is looked at again,
// scaled by a power of two: values up to the type's largest have a norm.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "quotient.cuh"

namespace moe {
namespace {

// (Blocks an SM, 5001 x 1407 fp32 with dsum: 4 / 5 / 6 27.6 / 25.2 / 29.2 us; three fit of the rows of 4096 bf16, 113 us, 126 with two.)
constexpr int kGradBlocksPerSm = 5, kGradBlocks = kGradBlocksPerSm * 152;   // most blocks of the gradient, each with a row of the workspace

// A piece as it lies in memory: N values (16 bytes of the rows' type) or one, unpacked where they are used.
template <class E, bool kVec, int N>
struct Raw {
    static constexpr int kWords = kVec ? N * static_cast<int>(sizeof(E)) / 4 : 1;
    uint32_t w[kWords];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const E* p)
    {
        if constexpr (kVec && kWords >= 4) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 q = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = q.x;
                w[4 * i + 1] = q.y;
                w[4 * i + 2] = q.z;
                w[4 * i + 3] = q.w;
            }
        } else if constexpr (kVec) {   // bf16 weights beside fp32 rows
            static_assert(!kVec || kWords >= 4 || kWords == 2, "8 bytes");
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            w[0] = q.x;
            w[kWords - 1] = q.y;
        } else if constexpr (sizeof(E) == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ __forceinline__ void put(E* p) const
    {
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (sizeof(E) == 4) {
            *reinterpret_cast<uint32_t*>(p) = w[0];
        } else {
            *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
        }
    }
    // the sums, rounded to the type
    __device__ __forceinline__ Raw plus(const Raw& o) const
    {
        Raw r;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(E) == 4)
                r.w[i] = __float_as_uint(at(i) + o.at(i));
            else if constexpr (kVec)
                r.w[i] = pack_bf16x2(at(2 * i) + o.at(2 * i), at(2 * i + 1) + o.at(2 * i + 1));
            else
                r.w[i] = pack_bf16x2(at(0) + o.at(0), 0.0f);
        }
        return r;
    }
    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (sizeof(E) == 4) return __uint_as_float(w[i]);
        return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};
template <class E, bool kVec, int N>
__device__ __forceinline__ void store(E* p, const float (&v)[N])
{
    if constexpr (sizeof(E) == 4) {
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
                reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
            *p = v[0];
        }
    } else if constexpr (kVec) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                                  pack_bf16x2(v[6], v[7]));
    } else {
        *p = __float2bfloat16_rn(v[0]);
    }
}
// weights of one type or the other, or ones
template <bool kVec, int N>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int at, float (&v)[N])
{
    if (!w) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 1.0f;
    } else if (f32) {
        Raw<float, kVec, N> r;
        r.load(static_cast<const float*>(w) + at);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = r.at(i);
    } else {
        Raw<__nv_bfloat16, kVec, N> r;
        r.load(static_cast<const __nv_bfloat16*>(w) + at);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = r.at(i);
    }
}

__device__ __forceinline__ uint16_t two_codes(float lo, float hi)
{
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(hi), "f"(lo));
    return two;
}

// A barrier of the W warps of a row (of one warp none), or of the block's rows together.  Rows of the gradient go their own
// ways, so that none does anything for a neighbour's sake (67000 x 1000 bf16 138 us, together 147); those of the forward,
// which have a block's start and end in common, go together (79.5 us, apart 82.6).
template <int W, bool kApart>
__device__ __forceinline__ void sync_row(int row_of)
{
    if (W >= 8 || (W > 1 && !kApart))
        __syncthreads();
    else if (W > 1)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + row_of), "n"(32 * W) : "memory");
}

// Sums (or maxima) over the W warps of a row, in every lane: the same order on every lane and call.  `buf` holds W
// values of the row's.
template <int W, bool kMax, bool kApart>
__device__ __forceinline__ float reduce(float v, float* buf, int row_of, int warp_of_row, int lane)
{
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = kMax ? fmaxf(v, o) : v + o;
    }
    if (W == 1) return v;
    if (lane == 0) buf[warp_of_row] = v;
    sync_row<W, kApart>(row_of);
    v = buf[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v = kMax ? fmaxf(v, buf[i]) : v + buf[i];
    return v;
}

// What multiplies the row: u = (s f) r, with f a power of two (1 but for rows whose squares overflow).
struct Scale {
    float f, r;
    bool finite;
};

// By the row's warps; where rows go together by all of the block, an ordinary row's result is what it was.  Leaves `buf` in use.
template <int W, int P, int N, bool kApart, class R>
__device__ __forceinline__ Scale scale_of(const R (&s)[P], float mean, float inv_cols, float eps, float* buf, int row_of, int warp_of_row, int lane)
{
    Scale o;
    float amax = 0.0f;
    bool nan = false;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float v = s[p].at(i);
            amax = fmaxf(amax, fabsf(v));
            nan = nan || v != v;
        }
    amax = reduce<W, true, kApart>(nan ? INFINITY : amax, buf, row_of, warp_of_row, lane);
    o.finite = amax < INFINITY;
    o.f = !(mean < INFINITY) && o.finite ? 0x1p-96f : 1.0f;
    float again = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i) again = fmaf(s[p].at(i) * o.f, s[p].at(i) * o.f, again);
    sync_row<W, kApart>(row_of);   // the maxima are read
    again = reduce<W, false, kApart>(again, buf, row_of, warp_of_row, lane);
    // (of eps, as of the squares, what f^2 leaves: as a rule nothing)
    o.r = o.finite ? __frsqrt_rn(fmaf(again, inv_cols, eps * o.f * o.f)) : NAN;
    return o;
}

// ---------------------------------------------------------------- forward

template <class T, bool kVec, int W, int P>
__global__ void __launch_bounds__(W >= 8 ? 32 * W : 256) rms_norm_kernel(const NormArgs a)
{
    constexpr int N = kVec ? 16 / static_cast<int>(sizeof(T)) : 1;
    constexpr int kRows = W >= 8 ? 1 : 8 / W;
    __shared__ float s_buf[3][kRows * W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row_of = warp / W, in_row = warp - row_of * W;
    const long long row = static_cast<long long>(blockIdx.x) * kRows + row_of;
    const bool live = row < a.rows;
    const int units = kVec ? a.cols / N : a.cols, first = in_row * 32 + lane;
    const T* const x = static_cast<const T*>(a.x) + (live ? row * a.x_stride : 0);
    const T* const res = static_cast<const T*>(a.residual) + (live && a.residual ? row * a.residual_stride : 0);

    Raw<T, kVec, N> s[P];
    float sum = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int u = first + p * 32 * W;
        s[p].clear();
        if (live && u < units) s[p].load(x + u * N);
    }
    if (a.residual) {
        Raw<T, kVec, N> r[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int u = first + p * 32 * W;
            r[p].clear();
            if (live && u < units) r[p].load(res + u * N);
        }
        T* const out = static_cast<T*>(a.sum) + (live && a.sum ? row * a.sum_stride : 0);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int u = first + p * 32 * W;
            // the residual stream is kept in the rows' type, and the norm is of what is kept: the gradient sees the same values
            s[p] = s[p].plus(r[p]);
            if (a.sum && live && u < units) s[p].put(out + u * N);
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i) sum = fmaf(s[p].at(i), s[p].at(i), sum);
    sum = reduce<W, false, false>(sum, s_buf[0] + row_of * W, row_of, in_row, lane);
    Scale scale{1.0f, 0.0f, true};
    const float mean = fmaf(sum, a.inv_cols, a.eps);
    const bool odd = !(mean < INFINITY);
    // (a row to itself is agreed on by all its warps; of several in a block each has to take part)
    if (W == 1 ? __any_sync(0xffffffffu, odd) : (W >= 8 ? odd : __syncthreads_or(odd) != 0))
        scale = scale_of<W, P, N, false>(s, mean, a.inv_cols, a.eps, s_buf[1] + row_of * W, row_of, in_row, lane);
    else
        scale.r = __frsqrt_rn(mean);
    if (!live && W > 1 && !a.codes) return;
    if (live && !scale.finite && first == 0) record_error(a.status, MOE_ERR_NONFINITE);

    // y of a piece; computed again for the codes, so that a lane holds its pieces as they lie in memory
    auto outputs = [&](int p, int u, float (&y)[N]) {
        float w[N];
        load_weight<kVec, N>(a.weight, a.weight_f32, u * N, w);
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = s[p].at(i) * scale.f * scale.r * w[i];
    };
    float amax = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int u = first + p * 32 * W;
        if (live && u < units) {
            float y[N];
            outputs(p, u, y);
#pragma unroll
            for (int i = 0; i < N; ++i) amax = fmaxf(amax, fabsf(y[i]));
            if (a.y) store<T, kVec, N>(static_cast<T*>(a.y) + row * a.y_stride + u * N, y);
        }
    }
    if (!a.codes) return;
    amax = reduce<W, true, false>(amax, s_buf[2] + row_of * W, row_of, in_row, lane);
    if (!live) return;
    // the scale of moe_quantize_fp8 (one rounding from fp32 to a code; the rounded y is not looked at again)
    const float sc = !scale.finite ? NAN : (amax > 0.0f ? amax / 448.0f : 1.0f);
    if (first == 0) a.scales[row] = sc;
    const float inv = sc >= kFmaDivMin ? __frcp_rn(sc) : 0.0f;
    uint8_t* const to = a.codes + row * a.codes_stride;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int u = first + p * 32 * W;
        if (u >= units) continue;
        float y[N], q[N];
        outputs(p, u, y);
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = inv != 0.0f ? div_by(y[i], sc, inv) : __fdiv_rn(y[i], sc);
        if constexpr (N == 8) {
            const uint32_t lo = two_codes(q[0], q[1]) | static_cast<uint32_t>(two_codes(q[2], q[3])) << 16;
            const uint32_t hi = two_codes(q[4], q[5]) | static_cast<uint32_t>(two_codes(q[6], q[7])) << 16;
            *reinterpret_cast<uint2*>(to + u * N) = make_uint2(lo, hi);
        } else if constexpr (N == 4) {
            *reinterpret_cast<uint32_t*>(to + u * N) = two_codes(q[0], q[1]) | static_cast<uint32_t>(two_codes(q[2], q[3])) << 16;
        } else {
            to[u] = static_cast<uint8_t>(two_codes(q[0], 0.0f));
        }
    }
}

// ---------------------------------------------------------------- gradient

// Blocks an SM that the gradient's registers are held to: 80 for pieces of eight bf16 values, of which a lane sums as many
// weights' gradients, 64 for four of fp32.  Measured for rows of 4096 bf16 and of 1407 fp32; elsewhere what follows from the
// same registers, at the cost of spills (rows of 8 to 2048 bf16, 56 to 152 bytes) or, from 4104 bf16 values on, of one block alone.
template <class T, bool kVec, int W, int P>
constexpr int grad_blocks()
{
    if (!kVec && W == 8 && P == 6 && sizeof(T) == 4) return kGradBlocksPerSm;
    if (!kVec && sizeof(T) == 2) return W <= 8 ? 3 : (W == 16 ? 2 : 1);
    return kVec && sizeof(T) == 2 ? (W <= 8 ? 3 : 1) : (W <= 8 ? 4 : (W == 16 ? 2 : 1));
}

template <class T, class D, bool kVec, int W, int P>
__global__ void __launch_bounds__(W >= 8 ? 32 * W : 256, (grad_blocks<T, kVec, W, P>())) rms_norm_backward_kernel(const NormGradArgs a)
{
    constexpr int N = kVec ? 16 / static_cast<int>(sizeof(T)) : 1;
    constexpr int kRows = W >= 8 ? 1 : 8 / W;
    __shared__ float2 s_sums[2][kRows * W];
    __shared__ float s_buf[kRows * W];
    __shared__ float s_dw[kRows > 1 ? (kRows - 1) * 32 * W * P * N : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row_of = warp / W, in_row = warp - row_of * W;
    const int units = kVec ? a.cols / N : a.cols, first = in_row * 32 + lane;
    let_next_start();

    float dw[P][N];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i) dw[p][i] = 0.0f;
    int turn = 0;
    // Rows of single bf16 values ask for the next row before they work on this one: 9000 x 1500 with dsum 52 us, 95 without (3000 x
    // 3001 41 and 36); 5001 x 1407 of fp32, whose blocks hide more of each other's waits, 37.6 us and 25.2.
    constexpr bool kAhead = !kVec && sizeof(T) == 2;
    Raw<T, kVec, N> next_s[P], next_d[P];
    Raw<D, kVec, N> next_g[P];
    auto fetch = [&](long long row, Raw<T, kVec, N> (&s)[P], Raw<D, kVec, N> (&g)[P], Raw<T, kVec, N> (&d)[P]) {
        const bool live = row < a.rows;
        const T* const x = static_cast<const T*>(a.x) + (live ? row * a.x_stride : 0);
        const D* const dy = static_cast<const D*>(a.dy) + (live ? row * a.dy_stride : 0);
        const T* const dsum = static_cast<const T*>(a.dsum) + (live && a.dsum ? row * a.dsum_stride : 0);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int u = first + p * 32 * W;
            s[p].clear();
            g[p].clear();
            d[p].clear();
            if (live && u < units) {
                s[p].load(x + u * N);
                g[p].load(dy + u * N);
                if (a.dsum) d[p].load(dsum + u * N);
            }
        }
    };
    if (kAhead) fetch(static_cast<long long>(blockIdx.x) * kRows + row_of, next_s, next_g, next_d);
    for (long long row0 = static_cast<long long>(blockIdx.x) * kRows; row0 < a.rows; row0 += static_cast<long long>(gridDim.x) * kRows) {
        const long long row = row0 + row_of;
        const bool live = row < a.rows;
        Raw<T, kVec, N> s[P], d[P];
        Raw<D, kVec, N> g[P];
        if (!kAhead) {
            fetch(row, s, g, d);
        } else {
#pragma unroll
            for (int p = 0; p < P; ++p) s[p] = next_s[p], g[p] = next_g[p], d[p] = next_d[p];
            fetch(row + static_cast<long long>(gridDim.x) * kRows, next_s, next_g, next_d);
        }
        // sum of s^2 and of w dy s, in one exchange between the warps
        float2 sums = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int u = first + p * 32 * W;
            if (u >= units) continue;
            float w[N];
            load_weight<kVec, N>(a.weight, a.weight_f32, u * N, w);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float v = s[p].at(i);
                sums.x = fmaf(v, v, sums.x);
                sums.y = fmaf(g[p].at(i) * w[i], v, sums.y);
            }
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            sums.x += __shfl_xor_sync(0xffffffffu, sums.x, off);
            sums.y += __shfl_xor_sync(0xffffffffu, sums.y, off);
        }
        if (W > 1) {
            // (two buffers in turn: a row's sums are read while another warp may be at the next row's)
            float2* const buf = s_sums[turn] + row_of * W;
            if (lane == 0) buf[in_row] = sums;
            sync_row<W, true>(row_of);
            sums = buf[0];
#pragma unroll
            for (int i = 1; i < W; ++i) {
                sums.x += buf[i].x;
                sums.y += buf[i].y;
            }
            turn ^= 1;
        }
        float f = 1.0f, r, dot = sums.y;
        const float mean = fmaf(sums.x, a.inv_cols, a.eps);
        const bool odd = !(mean < INFINITY) || !(fabsf(dot) < INFINITY);
        if (W == 1 ? __any_sync(0xffffffffu, odd) : odd) {   // (a row's lanes have the same sums)
            float* const buf = s_buf + row_of * W;
            const Scale scale = scale_of<W, P, N, true>(s, mean, a.inv_cols, a.eps, buf, row_of, in_row, lane);
            f = scale.f;
            r = scale.r;
            dot = 0.0f;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int u = first + p * 32 * W;
                if (u >= units) continue;
                float w[N];
                load_weight<kVec, N>(a.weight, a.weight_f32, u * N, w);
#pragma unroll
                for (int i = 0; i < N; ++i) dot = fmaf(g[p].at(i) * w[i], s[p].at(i) * f * r, dot);
            }
            sync_row<W, true>(row_of);   // (what scale_of left has been read)
            dot = reduce<W, false, true>(dot, buf, row_of, in_row, lane) * a.inv_cols;
            sync_row<W, true>(row_of);
        } else {
            r = __frsqrt_rn(mean);
            dot *= r * a.inv_cols;
        }
        T* const dx = static_cast<T*>(a.dx) + (live ? row * a.dx_stride : 0);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int u = first + p * 32 * W;
            if (u >= units) continue;
            float w[N], out[N];
            load_weight<kVec, N>(a.weight, a.weight_f32, u * N, w);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float unit = s[p].at(i) * f * r, gy = g[p].at(i);
                dw[p][i] = fmaf(gy, unit, dw[p][i]);
                out[i] = fmaf(f * r, fmaf(-unit, dot, gy * w[i]), d[p].at(i));
            }
            if (live) store<T, kVec, N>(dx + u * N, out);
        }
    }
    if (!a.dweight) return;
    // the block's rows that went side by side, then its row of the workspace
    if (kRows > 1) {
        if (row_of > 0)
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < N; ++i) s_dw[((row_of - 1) * P * N + p * N + i) * 32 * W + first] = dw[p][i];
        __syncthreads();
        if (row_of > 0) return;
        for (int o = 0; o < kRows - 1; ++o)
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < N; ++i) dw[p][i] += s_dw[(o * P * N + p * N + i) * 32 * W + first];
    }
    float* const part = a.parts + static_cast<long long>(blockIdx.x) * a.cols;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int u = first + p * 32 * W;
        if (u < units) store<float, kVec, N>(part + u * N, dw[p]);
    }
}

// dw[c] = the sum of the blocks' parts: 32 columns a block, 32 warps that take every 32nd part.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) rms_norm_weight_sum_kernel(const float* __restrict__ parts, int n, int cols,
                                                                           float* __restrict__ dw)
{
    __shared__ float s_sum[kSumWarps][32];
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < cols)
#pragma unroll 10
        for (int i = warp; i < n; i += kSumWarps) v += parts[static_cast<long long>(i) * cols + c];
    s_sum[warp][lane] = v;
    __syncthreads();
    if (warp > 0 || c >= cols) return;
    for (int i = 1; i < kSumWarps; ++i) v += s_sum[i][lane];
    dw[c] = v;
}

// ---------------------------------------------------------------- launches

template <class T, bool kVec, int W, int P>
void forward(const NormArgs& a, cudaStream_t s)
{
    constexpr int kRows = W >= 8 ? 1 : 8 / W;
    const unsigned grid = static_cast<unsigned>((a.rows + kRows - 1) / kRows);
    rms_norm_kernel<T, kVec, W, P><<<grid, W >= 8 ? 32 * W : 256, 0, s>>>(a);
}

template <class T, class D, bool kVec, int W, int P>
int backward(const NormGradArgs& a, cudaStream_t s)
{
    constexpr int kRows = W >= 8 ? 1 : 8 / W;
    const long long most = std::min(grad_blocks<T, kVec, W, P>() * num_sms(), kGradBlocks);
    const int grid = static_cast<int>(std::min<long long>((a.rows + kRows - 1) / kRows, most));
    rms_norm_backward_kernel<T, D, kVec, W, P><<<grid, W >= 8 ? 32 * W : 256, 0, s>>>(a);
    return grid;
}

// Warps and pieces for a row of this many units: as few warps as take it at two pieces a lane, past 8 warps at four and
// more (single values: six to eight a lane, and sixteen).
static_assert(kMaxNormCols <= 16384, "what the largest variants hold");
template <class T, class F>
auto by_size(bool vec, int units, F&& f)
{
    const auto go = [&](auto v, auto w, auto p) { return f(v, w, p); };
    using std::integral_constant;
    if (vec) {
        constexpr std::true_type v{};
        if (units <= 64) return go(v, integral_constant<int, 1>{}, integral_constant<int, 2>{});
        if (units <= 128) return go(v, integral_constant<int, 2>{}, integral_constant<int, 2>{});
        if (units <= 256) return go(v, integral_constant<int, 4>{}, integral_constant<int, 2>{});
        if (units <= 512) return go(v, integral_constant<int, 8>{}, integral_constant<int, 2>{});
        if (units <= 1024) return go(v, integral_constant<int, 16>{}, integral_constant<int, 2>{});
        if constexpr (kMaxNormCols * sizeof(T) / 16 > 2048) {   // (bf16 rows have no more)
            if (units > 2048) return go(v, integral_constant<int, 32>{}, integral_constant<int, 4>{});
        }
        return go(v, integral_constant<int, 16>{}, integral_constant<int, 4>{});
    }
    constexpr std::false_type v{};
    if (units <= 256) return go(v, integral_constant<int, 1>{}, integral_constant<int, 8>{});
    if (units <= 1024) return go(v, integral_constant<int, 4>{}, integral_constant<int, 8>{});
    if (units <= 1536) return go(v, integral_constant<int, 8>{}, integral_constant<int, 6>{});
    if (units <= 2048) return go(v, integral_constant<int, 8>{}, integral_constant<int, 8>{});
    if (units <= 3584) return go(v, integral_constant<int, 16>{}, integral_constant<int, 7>{});
    if (units <= 8192) return go(v, integral_constant<int, 32>{}, integral_constant<int, 8>{});
    return go(v, integral_constant<int, 32>{}, integral_constant<int, 16>{});
}

bool on(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

size_t rms_norm_ws_bytes(int cols)
{
    return cols > 0 && cols <= kMaxNormCols ? static_cast<size_t>(kGradBlocks) * cols * 4 : 0;
}

cudaError_t launch_rms_norm(NormArgs a, cudaStream_t s)
{
    if (a.rows <= 0) return cudaSuccess;
    a.inv_cols = 1.0f / static_cast<float>(a.cols);
    const int n = a.bf16 ? 8 : 4;
    bool vec = a.cols % n == 0 && on(a.weight, 16);
    for (const void* p : {a.x, a.residual, static_cast<const void*>(a.sum), static_cast<const void*>(a.y)}) vec = vec && on(p, 16);
    for (long long st : {a.x_stride, a.residual_stride, a.sum_stride, a.y_stride, a.codes_stride})
        vec = vec && (a.rows == 1 || st % n == 0);
    vec = vec && on(a.codes, n);
    const auto run = [&](auto type) {
        using T = decltype(type);
        by_size<T>(vec, vec ? a.cols / n : a.cols,
                   [&](auto v, auto w, auto p) { forward<T, decltype(v)::value, decltype(w)::value, decltype(p)::value>(a, s); });
    };
    a.bf16 ? run(__nv_bfloat16{}) : run(0.0f);
    return cudaGetLastError();
}

cudaError_t launch_rms_norm_backward(NormGradArgs a, cudaStream_t s)
{
    if (a.rows <= 0) return a.dweight ? cudaMemsetAsync(a.dweight, 0, static_cast<size_t>(a.cols) * 4, s) : cudaSuccess;
    a.inv_cols = 1.0f / static_cast<float>(a.cols);
    const int n = a.bf16 ? 8 : 4;
    bool vec = a.cols % n == 0 && on(a.weight, 16);
    for (const void* p : {a.x, a.dy, a.dsum, static_cast<const void*>(a.dx)}) vec = vec && on(p, 16);
    for (long long st : {a.x_stride, a.dy_stride, a.dsum_stride, a.dx_stride}) vec = vec && (a.rows == 1 || st % n == 0);
    const auto run = [&](auto type, auto dy_type) {
        using T = decltype(type);
        return by_size<T>(vec, vec ? a.cols / n : a.cols, [&](auto v, auto w, auto p) {
            return backward<T, decltype(dy_type), decltype(v)::value, decltype(w)::value, decltype(p)::value>(a, s);
        });
    };
    const __nv_bfloat16 b16{};
    const int grid = !a.bf16 ? run(0.0f, 0.0f) : (a.dy_f32 ? run(b16, 0.0f) : run(b16, b16));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.dweight) return e;
    return launch_after(rms_norm_weight_sum_kernel, dim3(static_cast<unsigned>((a.cols + 31) / 32)), 32 * kSumWarps, 0, s, a.parts, grid,
                        a.cols, a.dweight);
}

}  // namespace moe
