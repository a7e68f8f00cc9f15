// kv_append.cu -- the position rotation of q and k and the write of k and v
// into the paged cache, in one launch.
//
// Per token: n_heads + 2 n_kv_heads rows of D values, all read and written once.
// A row is D/16 lanes of two 16-byte pieces; the pieces of a lane are the two
// halves of its rotated pairs, so the rotation needs no exchange between lanes, and
// the e4m3 row maximum only one over the row's lanes.  A warp takes a token (or a
// part of its rows, when tokens are few): it computes the token's cosines and sines
// once, one or two a lane (a lane doing the eight that it needs cost more than the
// copies), and hands them around in shared memory.  A warp's rows arrive through a
// ring of its own in shared memory, some KB ahead of the writes and before the
// token's page and angles are known; held in registers they were too few in flight
// (72 us for 16384 tokens of 32 + 8 + 8 heads, D = 128; 63.5 us like this, 403 MB
// at 0.93 of the copy rate).
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

// Groups of rows that a warp has in its ring: 3 at 32 warps an SM; with more, warps or groups, reads and writes get in
// each other's way in memory (16384 tokens: 63.5 us, 40 warps 65; in blocks of 8 warps 5 groups 67, 6 groups 69; 48682
// tokens of 15 + 3 + 3 heads: 99 us, 4 groups 104, 40 warps 105).
constexpr int kDepth = 3;
// Warps work alone; small blocks free their places sooner (8 warps a block: 65 us instead of 63.5; 76622 tokens of 3 + 3 +
// 3 heads 95 and 86).
constexpr int kWarps = 2;

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

// Eight e4m3 codes of x * inv (inv a power of two: one rounding, to nearest even; NaN stays NaN).
__device__ __forceinline__ uint2 codes8(const Piece& p, float inv)
{
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t two;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(p.x[2 * i + 1] * inv), "f"(p.x[2 * i] * inv));
        w[i >> 1] |= static_cast<uint32_t>(two) << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

// The largest |x| of a row, one shuffle per halving of its kLanes lanes (NaN does not count).
template <int kLanes>
__device__ __forceinline__ float row_max(const Piece& x0, const Piece& x1)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(x0.x[i]), fabsf(x1.x[i])));
#pragma unroll
    for (int off = kLanes / 2; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
}

template <int D, bool kE4m3, bool kInterleaved>
__global__ void __launch_bounds__(32 * kWarps, 32 / kWarps) kv_append_kernel(const AppendArgs a)
{
    constexpr int kLanes = D / 16;          // lanes per row
    constexpr int kRows = 32 / kLanes;      // rows of a warp at a time
    extern __shared__ __align__(16) unsigned char smem[];   // [kWarps][kDepth] rings, then the angles
    float2(*const s_angle)[D / 2] = reinterpret_cast<float2(*)[D / 2]>(smem + kWarps * kDepth * 1024);
    const int lane = threadIdx.x & 31;
    const long long warp = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (warp >= static_cast<long long>(a.T) * a.parts) return;
    const int t = a.parts == 1 ? static_cast<int>(warp) : static_cast<int>(warp / a.parts);
    const int part = a.parts == 1 ? 0 : static_cast<int>(warp - static_cast<long long>(t) * a.parts);
    const int j = lane % kLanes, sub = lane / kLanes;
    const int pair_lanes = a.rot_dim / 16;
    // the lane's two pieces: the first one's place, and the second's behind it, in values
    const bool halves = !kInterleaved && j < pair_lanes;
    const int p0 = halves ? 8 * j : 16 * j, p1 = halves ? 8 * pair_lanes : 8;

    // the token's rows: heads of q, of k, of v; a row's place is its kind's base plus head * stride
    const int kv0 = a.n_heads, v0 = kv0 + a.n_kv_heads, rows = v0 + a.n_kv_heads, step = a.parts * kRows;
    const __nv_bfloat16* const q_row = a.q + t * a.q_token_stride + p0;
    const __nv_bfloat16* const k_row = a.k + t * a.k_token_stride + p0;
    const __nv_bfloat16* const v_row = a.v + t * a.v_token_stride + p0;
    const uint32_t ring = smem_u32(smem) + (threadIdx.x >> 5) * kDepth * 1024 + lane * 16;
    // the lane's pieces of row r0 + sub to their slot (a lane reads back what it copied itself)
    auto read = [&](int r0, uint32_t slot) {
        const int r = r0 + sub;
        if (r < rows) {
            const __nv_bfloat16* src = r < kv0 ? q_row : r < v0 ? k_row : v_row;
            src += static_cast<long long>(r < kv0 ? r : r < v0 ? r - kv0 : r - v0) *
                   (r < kv0 ? a.q_head : r < v0 ? a.k_head : a.v_head);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring + slot), "l"(src) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring + slot + 512), "l"(src + p1) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int n = 0; n < kDepth; ++n) read(part * kRows + n * step, n * 1024);

    // where the token's rows go in the cache, or nowhere
    const int pos = a.pos[t];
    const bool pad = pos < 0;
    long long place = -1, exp_place = 0;
    float2* const cs = s_angle[threadIdx.x >> 5];
    if (!pad) {   // the whole warp
        const int seq = a.seq ? a.seq[t] : t;
        const int pg = pos / a.page_size, at = pos - pg * a.page_size;
        if (seq >= 0 && seq < a.n_seqs && pg < a.max_pages) {
            const int e = a.page_table[seq * a.table_stride + pg];
            if (e >= 0 && e < a.n_pages) {
                place = e * a.page_stride + at * a.token_stride;
                if (kE4m3) exp_place = e * a.exp_page_stride + at * a.exp_token_stride;
            }
        }
        for (int i = lane; i < a.rot_dim / 2; i += 32) {
            float x, y;
            cos_sin_turn(a.phase[i] * static_cast<uint64_t>(static_cast<uint32_t>(pos)), x, y);
            cs[i] = make_float2(x, y);
        }
        if (place < 0 && lane == 0) record_error(a.status, MOE_ERR_INDEX);
    }
    __syncwarp();
    const float4* const mine = reinterpret_cast<const float4*>(cs + 8 * j);   // of the lane's eight pairs
    constexpr int kElt = kE4m3 ? 1 : 2;
    __nv_bfloat16* const q_to = a.q_out + t * a.q_out_token_stride + p0;
    char* const k_to = static_cast<char*>(a.cache_k) + (place + p0) * kElt;
    char* const v_to = static_cast<char*>(a.cache_v) + (place + p0) * kElt;

    uint32_t slot = 0;
    for (int r0 = part * kRows; r0 < rows; r0 += step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        const int r = r0 + sub;
        const bool live = r < rows;   // whole rows: the lanes of a row agree
        const bool is_q = r < kv0, is_v = r >= v0;
        Piece x0{}, x1{};
        if (live && !pad) {
            uint4 w0, w1;
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w0.x), "=r"(w0.y), "=r"(w0.z), "=r"(w0.w) : "r"(ring + slot) : "memory");
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w1.x), "=r"(w1.y), "=r"(w1.z), "=r"(w1.w) : "r"(ring + slot + 512) : "memory");
            x0 = unpack(w0);
            x1 = unpack(w1);
        }
        if (j < pair_lanes && !pad && !is_v) {
            if (kInterleaved) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float4 w = mine[i / 2];
                    Piece& p = i < 4 ? x0 : x1;
                    const int k = 2 * (i & 3);
                    const float a0 = p.x[k], b0 = p.x[k + 1], a1 = p.x[k + 2], b1 = p.x[k + 3];
                    p.x[k] = a0 * w.x - b0 * w.y;
                    p.x[k + 1] = a0 * w.y + b0 * w.x;
                    p.x[k + 2] = a1 * w.z - b1 * w.w;
                    p.x[k + 3] = a1 * w.w + b1 * w.z;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float4 w = mine[i / 2];
                    const float a0 = x0.x[i], b0 = x1.x[i], a1 = x0.x[i + 1], b1 = x1.x[i + 1];
                    x0.x[i] = a0 * w.x - b0 * w.y;
                    x1.x[i] = a0 * w.y + b0 * w.x;
                    x0.x[i + 1] = a1 * w.z - b1 * w.w;
                    x1.x[i + 1] = a1 * w.w + b1 * w.z;
                }
            }
        }
        const int head = is_v ? r - v0 : r - kv0;
        const bool stored = live && !is_q && place >= 0;
        if (kE4m3) {
            float amax = row_max<kLanes>(x0, x1);
            if (__any_sync(0xffffffffu, !is_q && amax == INFINITY)) {   // infinities are stored as NaN and do not count
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x0.x[i] = is_q || fabsf(x0.x[i]) < INFINITY ? x0.x[i] : NAN;
                    x1.x[i] = is_q || fabsf(x1.x[i]) < INFINITY ? x1.x[i] : NAN;
                }
                amax = row_max<kLanes>(x0, x1);
            }
            if (stored) {
                // the smallest e with amax <= 448 * 2^e = 1.75 * 2^(8 + e)
                const uint32_t b = __float_as_uint(amax);
                int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
                e = amax == 0.0f ? 0 : max(e, -126);
                const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                char* dst = (is_v ? v_to : k_to) + static_cast<long long>(head) * a.cache_head;
                *reinterpret_cast<uint2*>(dst) = codes8(x0, inv);
                *reinterpret_cast<uint2*>(dst + p1) = codes8(x1, inv);
                if (j == 0) (is_v ? a.v_exp : a.k_exp)[exp_place + head * a.exp_head_stride] = static_cast<uint8_t>(e + 127);
            }
        }
        if ((live && is_q) || (!kE4m3 && stored)) {
            char* dst = is_q ? reinterpret_cast<char*>(q_to + static_cast<long long>(r) * a.q_out_head)
                             : (is_v ? v_to : k_to) + static_cast<long long>(head) * a.cache_head;
            *reinterpret_cast<uint4*>(dst) = pack(x0);
            *reinterpret_cast<uint4*>(dst + 2 * p1) = pack(x1);
        }
        read(r0 + kDepth * step, slot);
        slot = slot == (kDepth - 1) * 1024 ? 0 : slot + 1024;
    }
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, bool e4m3, cudaStream_t s)
{
    const long long warps = static_cast<long long>(a.T) * a.parts;
    const unsigned grid = static_cast<unsigned>((warps + kWarps - 1) / kWarps);
    constexpr int kSmem = kWarps * (kDepth * 1024 + D / 2 * 8);
    const auto kernel = e4m3 ? (a.interleaved ? kv_append_kernel<D, true, true> : kv_append_kernel<D, true, false>)
                             : (a.interleaved ? kv_append_kernel<D, false, true> : kv_append_kernel<D, false, false>);
    static_assert(kSmem <= 48 * 1024, "within the limit that needs no asking");
    kernel<<<grid, 32 * kWarps, kSmem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(AppendArgs a, int head_dim, bool e4m3, cudaStream_t s)
{
    if (a.T <= 0) return cudaSuccess;
    // One warp per token, more (down to kRows rows each) while the tokens alone do not fill the machine: 24 warps an SM in
    // all (32 + 8 + 8 heads, us with 1 / 2 / 4 / 12 warps a token: 8 tokens 6.9 / 5.2 / 4.0 / 3.1, 300 tokens 7.2 / 5.1 /
    // 4.2 / 4.1, 1000 tokens 7.2 / 7.0 / 7.0 / 8.6, 4000 tokens 20.0 / 20.9 / 25.5 / 32.1).
    const int groups = (a.n_heads + 2 * a.n_kv_heads + 512 / head_dim - 1) / (512 / head_dim);
    const int want = static_cast<int>((24LL * num_sms() + a.T - 1) / a.T);
    a.parts = want < 1 ? 1 : (want > groups ? groups : want);
    switch (head_dim) {
        case 64: return launch_d<64>(a, e4m3, s);
        case 128: return launch_d<128>(a, e4m3, s);
        default: return launch_d<256>(a, e4m3, s);
    }
}

}  // namespace moe
