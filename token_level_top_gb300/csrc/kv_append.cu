// kv_append.cu -- the position rotation of q and k and the write of k and v
// into the paged cache, in one launch.
//
// Per token: n_heads + 2 n_kv_heads rows of D values.  A row is D/16 lanes of
// two 16-byte pieces; the pieces of a lane are the two halves of its rotated
// pairs, so the rotation needs no exchange between lanes, and the e4m3 row
// maximum only one over the row's lanes.  A lane's eight angles depend on the
// token and the lane alone and are reused for every row that its warp takes.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

// cos and sin of 2 pi f / 2^64.  The angle arrives modulo a turn; the nearest
// quarter turn is taken off in integers, so the float argument (in half turns,
// at most 1/4) keeps full precision at every position.
__device__ __forceinline__ void cos_sin_turn(uint64_t f, float& c, float& s)
{
    const int32_t t = static_cast<int32_t>(f >> 32);                  // turns * 2^32
    const int32_t quarter = static_cast<int32_t>(static_cast<uint32_t>(t) + (1u << 29)) >> 30;   // -2 .. 1
    const int32_t r = static_cast<int32_t>(static_cast<uint32_t>(t) - (static_cast<uint32_t>(quarter) << 30));
    float sr, cr;
    sincospif(static_cast<float>(r) * 0x1p-31f, &sr, &cr);
    const bool swap = (quarter & 1) != 0;
    const float a = swap ? sr : cr, b = swap ? cr : sr;
    c = ((quarter + 1) & 2) ? -a : a;
    s = (quarter & 2) ? -b : b;
}

struct Piece {
    float x[8];
};

__device__ __forceinline__ Piece unpack(const uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    Piece p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p.x[2 * i] = __uint_as_float(w[i] << 16);
        p.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return p;
}

__device__ __forceinline__ uint4 pack(const Piece& p)
{
    return make_uint4(pack_bf16x2(p.x[0], p.x[1]), pack_bf16x2(p.x[2], p.x[3]), pack_bf16x2(p.x[4], p.x[5]),
                      pack_bf16x2(p.x[6], p.x[7]));
}

__device__ __forceinline__ float finite_abs(float x)
{
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.0f;   // NaN fails the comparison too
}

// Eight e4m3 codes of x * inv (inv a power of two: one rounding, to nearest even).
__device__ __forceinline__ uint2 codes8(const Piece& p, float inv)
{
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // a value that is not finite becomes NaN (the conversion would saturate an infinity)
        const float a = fabsf(p.x[2 * i]) < INFINITY ? p.x[2 * i] * inv : NAN;
        const float b = fabsf(p.x[2 * i + 1]) < INFINITY ? p.x[2 * i + 1] * inv : NAN;
        uint16_t two;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(b), "f"(a));
        w[i >> 1] |= static_cast<uint32_t>(two) << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

template <int D, bool kE4m3, bool kInterleaved>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a)
{
    constexpr int kLanes = D / 16;          // lanes per row
    constexpr int kRows = 32 / kLanes;      // rows of a warp at a time
    const int lane = threadIdx.x & 31;
    const long long warp = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (warp >= static_cast<long long>(a.T) * a.parts) return;
    const int t = static_cast<int>(warp / a.parts);
    const int part = static_cast<int>(warp - static_cast<long long>(t) * a.parts);
    const int j = lane % kLanes, sub = lane / kLanes;
    const int pos = a.pos[t];

    // where the token's rows go: page * page_stride + offset * token_stride, or nowhere
    long long page = -1;
    int at = 0;
    if (pos >= 0) {
        const int seq = a.seq ? a.seq[t] : t;
        const int pg = pos / a.page_size;
        at = pos - pg * a.page_size;
        if (seq >= 0 && seq < a.n_seqs && pg < a.max_pages) {
            const int e = a.page_table[seq * a.table_stride + pg];
            if (e >= 0 && e < a.n_pages) page = e;
        }
        if (page < 0 && lane == 0) record_error(a.status, MOE_ERR_INDEX);
    }

    const int pair_lanes = a.rot_dim / 16;
    const bool rotated = j < pair_lanes && pos >= 0;
    // the lane's two pieces, in units of 8 values
    int p0, p1;
    if (!kInterleaved && j < pair_lanes) {
        p0 = j;
        p1 = j + pair_lanes;
    } else {
        p0 = 2 * j;
        p1 = 2 * j + 1;
    }
    float c[8], s[8];
    if (rotated) {
        const ulonglong2* ph = reinterpret_cast<const ulonglong2*>(a.phase) + 4 * j;
        const uint64_t up = static_cast<uint32_t>(pos);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const ulonglong2 f = ph[i];
            cos_sin_turn(f.x * up, c[2 * i], s[2 * i]);
            cos_sin_turn(f.y * up, c[2 * i + 1], s[2 * i + 1]);
        }
    }

    const int rows = a.n_heads + 2 * a.n_kv_heads;
    for (int r0 = part * kRows; r0 < rows; r0 += a.parts * kRows) {
        const int r = r0 + sub;
        const bool live = r < rows;   // whole rows: the lanes of a row agree
        const bool is_q = r < a.n_heads, is_v = r >= a.n_heads + a.n_kv_heads;
        const int head = is_q ? r : (is_v ? r - a.n_heads - a.n_kv_heads : r - a.n_heads);
        Piece x0{}, x1{};
        if (live && pos >= 0) {
            const __nv_bfloat16* src =
                is_q ? a.q + t * a.q_token_stride + head * a.q_head_stride
                     : (is_v ? a.v + t * a.v_token_stride + head * a.v_head_stride
                             : a.k + t * a.k_token_stride + head * a.k_head_stride);
            x0 = unpack(*reinterpret_cast<const uint4*>(src + 8 * p0));
            x1 = unpack(*reinterpret_cast<const uint4*>(src + 8 * p1));
        }
        if (rotated && !is_v) {
            if (kInterleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    Piece& p = i < 4 ? x0 : x1;
                    const float u = p.x[2 * (i & 3)], w = p.x[2 * (i & 3) + 1];
                    p.x[2 * (i & 3)] = u * c[i] - w * s[i];
                    p.x[2 * (i & 3) + 1] = u * s[i] + w * c[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = x0.x[i], w = x1.x[i];
                    x0.x[i] = u * c[i] - w * s[i];
                    x1.x[i] = u * s[i] + w * c[i];
                }
            }
        }
        if (live && is_q) {
            __nv_bfloat16* dst = a.q_out + t * a.q_out_token_stride + head * a.q_out_head_stride;
            *reinterpret_cast<uint4*>(dst + 8 * p0) = pack(x0);
            *reinterpret_cast<uint4*>(dst + 8 * p1) = pack(x1);
        }
        if (kE4m3) {
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(finite_abs(x0.x[i]), finite_abs(x1.x[i])));
#pragma unroll
            for (int off = kLanes / 2; off >= 1; off >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            if (live && !is_q && page >= 0) {
                // the smallest e with amax <= 448 * 2^e = 1.75 * 2^(8 + e)
                const uint32_t b = __float_as_uint(amax);
                int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
                e = amax == 0.0f ? 0 : max(e, -126);
                const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                uint8_t* dst = static_cast<uint8_t*>(is_v ? a.cache_v : a.cache_k) + page * a.page_stride +
                               at * a.token_stride + head * a.head_stride;
                *reinterpret_cast<uint2*>(dst + 8 * p0) = codes8(x0, inv);
                *reinterpret_cast<uint2*>(dst + 8 * p1) = codes8(x1, inv);
                if (j == 0)
                    (is_v ? a.v_exp : a.k_exp)[page * a.exp_page_stride + at * a.exp_token_stride +
                                               head * a.exp_head_stride] = static_cast<uint8_t>(e + 127);
            }
        } else if (live && !is_q && page >= 0) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? a.cache_v : a.cache_k) + page * a.page_stride +
                                 at * a.token_stride + head * a.head_stride;
            *reinterpret_cast<uint4*>(dst + 8 * p0) = pack(x0);
            *reinterpret_cast<uint4*>(dst + 8 * p1) = pack(x1);
        }
    }
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, bool e4m3, cudaStream_t s)
{
    const long long warps = static_cast<long long>(a.T) * a.parts;
    const unsigned grid = static_cast<unsigned>((warps + 7) / 8);
    if (e4m3) {
        if (a.interleaved)
            kv_append_kernel<D, true, true><<<grid, 256, 0, s>>>(a);
        else
            kv_append_kernel<D, true, false><<<grid, 256, 0, s>>>(a);
    } else {
        if (a.interleaved)
            kv_append_kernel<D, false, true><<<grid, 256, 0, s>>>(a);
        else
            kv_append_kernel<D, false, false><<<grid, 256, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(AppendArgs a, int head_dim, bool e4m3, cudaStream_t s)
{
    if (a.T <= 0) return cudaSuccess;
    // one warp per token, more (down to one row group each) while the tokens
    // alone do not fill the machine
    const int groups = (a.n_heads + 2 * a.n_kv_heads + 512 / head_dim - 1) / (512 / head_dim);
    const int want = static_cast<int>((32LL * num_sms() + a.T - 1) / a.T);
    a.parts = want < 1 ? 1 : (want > groups ? groups : want);
    switch (head_dim) {
        case 64: return launch_d<64>(a, e4m3, s);
        case 128: return launch_d<128>(a, e4m3, s);
        default: return launch_d<256>(a, e4m3, s);
    }
}

}  // namespace moe
