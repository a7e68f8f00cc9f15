// attention.cu -- attention of one new token per sequence over the paged cache.
//
// The cache is read once, so the kernel is a stream of key and value rows
// (2 D elements per key and key head) with little arithmetic on top; its floor
// is the bytes of the live rows at the copy bandwidth.
//
// Work: the live keys of every (sequence, key head, block of query heads) are
// cut into granules of 16 keys per warp.  The granules of the whole batch, in
// that order, are dealt out in equal runs to one block per SM, whatever the
// lengths: each block finds its run from the lengths alone (a scan over them),
// so nothing is planned on the host and a captured graph follows the lengths.
// A run may end inside an item; such an item's parts (maximum, sum and
// unnormalised output) go to the workspace and the block that finishes last
// joins them, always in the same order.
//
// A warp's tile is 16 keys.  Every lane copies exactly the 16-byte pieces that
// it will feed to the matrix instructions (cp.async into its own place of a
// ring in shared memory), so the ring needs no barrier and no bank is hit
// twice, and some 100 to 190 KB per SM are in flight whatever the arithmetic does.
//   scores: C[head][key] = Q K^T, m16n8k16.  The inner dimension may be taken in
//   any order if both sides agree: a lane's 16 bytes of a key row are its B
//   fragments of consecutive steps, and the same 16 bytes of Q its A fragments.
//   values: C[head][d] += P V.  The C layout of the scores is the A layout of
//   the weights; a lane holds pieces of four keys' rows, which byte permutes
//   pair up into B fragments.
// The weights go in as the sum of two 16-bit parts (their own rounding would
// cost more than the output's): with at most 8 query heads the low parts use
// the other 8 rows of the same instruction.
//
// e4m3 rows become f16 in one conversion per two codes (exact), so that path
// multiplies in f16: Q is scaled by a power of two per head, and the value rows'
// exponents enter as 2^(s + e) in the weights, whose running maximum is taken
// over s + e; the sum of the softmax uses 2^s against the same maximum.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kAttentionCtas = 152;   // most blocks of a launch (one per SM)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// e4m3 path: weights are held times 2^14, so that f16 keeps those 2^-38 of the largest
constexpr float kShift = 14.0f;

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, bool f16)
{
    if (f16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Copies N bytes, or writes N zeros when !live (src is then not read).
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool live)
{
    const int n = live ? N : 0;
    if (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// The first n bytes of the 4 at src (4-byte aligned), zeros behind them.
__device__ __forceinline__ void copy_async_4(uint32_t dst, const void* src, int n)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// Two e4m3 codes (the low or high half of w) to two f16, exactly.
__device__ __forceinline__ uint32_t f16_of_codes(uint32_t w, int half)
{
    uint32_t r;
    const uint16_t two = static_cast<uint16_t>(half ? w >> 16 : w & 0xffffu);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// 2^(byte - 127); byte 0 is a subnormal.
__device__ __forceinline__ float pow2_of_byte(uint32_t b)
{
    return __uint_as_float(b ? b << 23 : 0x00400000u);
}

// (a, b) as the sum of two pairs of 16-bit values.
template <bool kF16>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo)
{
    if (kF16) {
        const __half2 h = __floats2half2_rn(a, b);
        const float2 back = __half22float2(h);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        lo = pack_f16x2(a - back.x, b - back.y);
    } else {
        hi = pack_bf16x2(a, b);
        lo = pack_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
    }
}

template <int D, bool kE4m3>
struct Shape {
    static constexpr int kRow = D * (kE4m3 ? 1 : 2);          // bytes of a row
    static constexpr int kWarps = D == 256 ? 4 : 8;          // at D = 256 a warp needs 255 registers
    static constexpr int kTile = 16 * kRow;                   // bytes of a warp's key (or value) tile
    static constexpr int kGranule = 16 * kWarps;              // keys
    static constexpr int kMerge = kWarps * 8 * D * 4;         // the block's join of 8 heads
    // beside a tile: which of its keys are live, and e4m3 32 exponent words and where their bytes are
    static constexpr int kMeta = kE4m3 ? 192 : 16, kMask = kE4m3 ? 128 : 0, kByte = 132;
    // as many stages as 227 KB hold beside the join, at most 8
    static constexpr int kFit = (232448 - 512 - kMerge - kWarps * 128) / (kWarps * (2 * kTile + kMeta));
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr int kRing = kWarps * kStages * 2 * kTile;
    static constexpr int kSmem = kRing + kMerge + kWarps * (kStages * kMeta + 128);
    static constexpr int kKeySegs = kRow / 64;                // 16-byte pieces of a key row per lane
    static constexpr int kValBytes = kRow / 8 < 16 ? kRow / 8 : 16;
    static constexpr int kValSegs = kRow / (8 * kValBytes);
    static constexpr int kValElts = kValBytes / (kE4m3 ? 1 : 2);
    static constexpr int kSteps = kE4m3 ? 4 : 2;              // inner steps per 16-byte piece
    static constexpr int kQ = D / 8;                          // A registers of one half of the heads
    static constexpr int kTiles = D / 8;                      // output column tiles
};

// One item of the work list while it is walked granule by granule.
struct Walk {
    int b, h;            // sequence; key head * head blocks + head block
    int len, first, n;   // its live keys [first, len) and its granules (per h)
    int g;               // granule within the item
    long long off;       // the item's first granule in the whole list
};

__device__ __forceinline__ int clamped_len(const AttentionArgs& a, int b, bool record)
{
    const long long most = static_cast<long long>(a.max_pages) * a.page_size;
    const int n = a.seq_len[b];
    if (n >= 0 && n <= most) return n;
    if (record) record_error(a.status, MOE_ERR_INDEX);
    return n < 0 ? 0 : static_cast<int>(most);
}

__device__ __forceinline__ int live_keys(const AttentionArgs& a, int len)
{
    return a.window > 0 && len > a.window ? a.window : len;
}

template <int kGranule>
__device__ __forceinline__ void load_item(const AttentionArgs& a, Walk& w)
{
    w.len = clamped_len(a, w.b, false);
    const int live = live_keys(a, w.len);
    w.first = w.len - live;
    w.n = (live + kGranule - 1) / kGranule;
}

// The next granule; past the end of the batch the walk stays on its last item.
template <int kGranule>
__device__ __forceinline__ void advance(const AttentionArgs& a, Walk& w, int heads)
{
    if (++w.g < w.n) return;
    w.off += w.n;
    w.g = 0;
    if (++w.h < heads) return;
    w.h = 0;
    do {
        if (++w.b >= a.B) {
            w.n = 0;
            return;
        }
        load_item<kGranule>(a, w);
    } while (w.n == 0);
}

// The e4m3 and bf16 paths differ in how bytes become fragments and in the weights.
template <int D, bool kE4m3, int kHeads>
__global__ void __launch_bounds__(32 * Shape<D, kE4m3>::kWarps, 1) paged_attention_kernel(const AttentionArgs a)
{
    using S = Shape<D, kE4m3>;
    constexpr int kWarps = S::kWarps, kThreads = 32 * kWarps, kStages = S::kStages;
    constexpr int kHalves = kHeads / 8;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long s_scan[kWarps];
    __shared__ Walk s_start;
    __shared__ int s_last;
    float* const s_merge = reinterpret_cast<float*>(smem + S::kRing);
    unsigned char* const s_meta = smem + S::kRing + S::kMerge;              // [warp][stage]
    float2* const s_ml = reinterpret_cast<float2*>(s_meta + kWarps * kStages * S::kMeta);   // [warp][16]

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int group = a.n_heads / a.n_kv_heads;                 // query heads per key head
    const int blocks = (group + kHeads - 1) / kHeads;           // head blocks per key head
    const int heads = a.n_kv_heads * blocks;                    // items per sequence

    // ---- the batch's granules, and where this block's run begins
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b)
        mine += (live_keys(a, clamped_len(a, b, blockIdx.x == 0)) + S::kGranule - 1) / S::kGranule;
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) s_scan[warp] = incl;
    // sequences without live keys: zeros
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (live_keys(a, clamped_len(a, b, false)) > 0) continue;
        for (int i = threadIdx.x; i < a.n_heads * (D / 8); i += kThreads) {
            const int h = i / (D / 8), d = i % (D / 8);
            *reinterpret_cast<uint4*>(a.out + b * a.out_token_stride + h * a.out_head_stride + 8 * d) = make_uint4(0, 0, 0, 0);
            if (a.lse && d == 0) a.lse[static_cast<long long>(b) * a.n_heads + h] = -INFINITY;
        }
    }
    __syncthreads();
    long long total = 0, before = incl - mine;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += s_scan[i];
        total += s_scan[i];
    }
    const long long all = total * heads;
    const long long run = (all + gridDim.x - 1) / gridDim.x;    // granules per block
    const long long lo = run * blockIdx.x, hi = min(all, lo + run);
    if (lo >= hi) return;
    if (mine > 0 && before * heads <= lo && lo < (before + mine) * heads) {
        Walk w{};
        w.b = b0;
        w.off = before * heads;
        load_item<S::kGranule>(a, w);
        while (w.off + static_cast<long long>(w.n) * heads <= lo) {
            w.off += static_cast<long long>(w.n) * heads;
            ++w.b;
            load_item<S::kGranule>(a, w);
        }
        w.h = static_cast<int>((lo - w.off) / w.n);
        w.off += static_cast<long long>(w.h) * w.n;
        w.g = static_cast<int>(lo - w.off);
        s_start = w;
    }
    __syncthreads();

    const uint32_t ring = smem_u32(smem) + warp * kStages * 2 * S::kTile;
    unsigned char* const meta = s_meta + warp * kStages * S::kMeta;
    Walk iw = s_start, cw = s_start;
    const int count = static_cast<int>(hi - lo);

    // ---- the copying side: key `lane & 15` of the tile belongs to this lane
    int next_page = -1, next_at = 0;
    bool next_live = false;
    auto look_up = [&]() {
        const int key = iw.first + iw.g * S::kGranule + warp * 16 + (lane & 15);
        next_live = iw.n > 0 && key < iw.len;
        if (next_live) {
            const int j = static_cast<int>(static_cast<unsigned>(key) / static_cast<unsigned>(a.page_size));
            next_at = key - j * a.page_size;
            next_page = __ldg(a.page_table + iw.b * a.table_stride + j);
        }
    };
    auto issue = [&](int stage) {
        const int hk = iw.h / blocks;
        bool live = next_live;
        long long row = 0;
        if (live) {
            if (next_page >= 0 && next_page < a.n_pages)
                row = next_page * a.page_stride + next_at * a.token_stride + hk * a.head_stride;
            else {
                record_error(a.status, MOE_ERR_INDEX);
                live = false;
            }
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, live);
        const uint32_t dst = ring + stage * 2 * S::kTile + lane * 16;
        const char* const kb = static_cast<const char*>(a.k);
        const char* const vb = static_cast<const char*>(a.v);
        constexpr int kElt = kE4m3 ? 1 : 2;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const long long r = __shfl_sync(0xffffffffu, row, t * 8 + g) * kElt + c * 16;
            const bool ok = (mask >> (t * 8 + g)) & 1;
#pragma unroll
            for (int u = 0; u < S::kKeySegs; ++u)
                copy_async<16>(dst + (t * S::kKeySegs + u) * 512, kb + r + u * 64, ok);
        }
        const uint32_t vdst = ring + stage * 2 * S::kTile + S::kTile + lane * S::kValBytes;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int key = 2 * c + (t & 1) + (t >> 1) * 8;
            const long long r = __shfl_sync(0xffffffffu, row, key) * kElt + g * S::kValBytes;
            const bool ok = (mask >> key) & 1;
#pragma unroll
            for (int u = 0; u < S::kValSegs; ++u)
                copy_async<S::kValBytes>(vdst + (t * S::kValSegs + u) * 32 * S::kValBytes, vb + r + u * 8 * S::kValBytes, ok);
        }
        if (kE4m3) {
            // lanes 0..15 fetch the keys' exponent bytes, 16..31 the values': the byte is the last of the
            // `n` copied ones of its aligned word, so nothing behind it is read
            const uint8_t* e = (lane < 16 ? a.k_exp : a.v_exp);
            int n = 0;
            if (live) {
                e += next_page * a.exp_page_stride + next_at * a.exp_token_stride + hk * a.exp_head_stride;
                n = static_cast<int>(reinterpret_cast<uintptr_t>(e) & 3) + 1;
                e -= n - 1;
            }
            copy_async_4(smem_u32(meta) + stage * S::kMeta + lane * 4, e, n);
            meta[stage * S::kMeta + S::kByte + lane] = static_cast<unsigned char>(n);
        }
        if (lane == 0) *reinterpret_cast<uint32_t*>(meta + stage * S::kMeta + S::kMask) = mask;
        advance<S::kGranule>(a, iw, heads);
        look_up();
    };

    look_up();
    for (int i = 0; i < kStages; ++i) {
        if (i < count) issue(i);
        copy_commit();
    }

    // ---- the computing side
    uint32_t q[kHalves][S::kQ];
    float qscale[kHalves];            // scores in units of log2: accumulator * qscale (* the key's exponent)
    float o[S::kTiles][4];
    float m[kHalves], l[kHalves];
    int stage = 0;
    for (int i = 0; i < count; ++i) {
        const int hk = cw.h / blocks, block = cw.h - hk * blocks;
        const int head0 = hk * group + block * kHeads, live_heads = min(kHeads, group - block * kHeads);
        if (i == 0 || cw.g == 0) {    // a new item
#pragma unroll
            for (int hh = 0; hh < kHalves; ++hh) {
                const bool ok = hh * 8 + g < live_heads;
                const __nv_bfloat16* src = a.q + cw.b * a.q_token_stride + (head0 + hh * 8 + g) * a.q_head_stride;
                m[hh] = -INFINITY;
                l[hh] = 0.0f;
                if (!kE4m3) {
#pragma unroll
                    for (int u = 0; u < S::kKeySegs; ++u) {
                        const uint4 v = ok ? *reinterpret_cast<const uint4*>(src + u * 32 + c * 8) : make_uint4(0, 0, 0, 0);
                        q[hh][4 * u] = v.x;
                        q[hh][4 * u + 1] = v.y;
                        q[hh][4 * u + 2] = v.z;
                        q[hh][4 * u + 3] = v.w;
                    }
                    qscale[hh] = a.scale * kLog2e;
                } else {
                    // bf16 to f16 after a power of two that puts the row's largest value near 2^13: values
                    // down to 2^-27 of it stay exact
                    uint4 v[2 * S::kKeySegs];
                    float top = 0.0f;
#pragma unroll
                    for (int u = 0; u < 2 * S::kKeySegs; ++u) {
                        v[u] = ok ? *reinterpret_cast<const uint4*>(src + (u >> 1) * 64 + c * 16 + (u & 1) * 8) : make_uint4(0, 0, 0, 0);
                        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x = fabsf(__uint_as_float(w[j] << 16)), y = fabsf(__uint_as_float(w[j] & 0xffff0000u));
                            top = fmaxf(top, x < INFINITY ? x : 0.0f);
                            top = fmaxf(top, y < INFINITY ? y : 0.0f);
                        }
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    int e = 13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
                    e = top == 0.0f ? 0 : max(-114, min(100, e));
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                    qscale[hh] = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                    for (int u = 0; u < 2 * S::kKeySegs; ++u) {
                        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            q[hh][4 * u + j] = pack_f16x2(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[t][j] = 0.0f;
        }

        copy_wait<kStages - 1>();
        __syncwarp();
        const uint32_t mask = *reinterpret_cast<const volatile uint32_t*>(meta + stage * S::kMeta + S::kMask);
        if (mask & 0xffffu) {
            const uint32_t kt = ring + stage * 2 * S::kTile + lane * 16;
            float s[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[t][j] = 0.0f;
#pragma unroll
            for (int u = 0; u < S::kKeySegs; ++u)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint4 v = lds128(kt + (t * S::kKeySegs + u) * 512);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < S::kSteps; ++k) {
                        const uint32_t k0 = kE4m3 ? f16_of_codes(w[k], 0) : w[2 * (k & 1)];
                        const uint32_t k1 = kE4m3 ? f16_of_codes(w[k], 1) : w[2 * (k & 1) + 1];
                        const int at = (u * S::kSteps + k) * 2;
                        mma_16816(s[t], q[0][at], kHalves == 2 ? q[kHalves - 1][at] : 0u, q[0][at + 1],
                                  kHalves == 2 ? q[kHalves - 1][at + 1] : 0u, k0, k1, kE4m3);
                    }
                }

            // scores to log2 units; keys 2c, 2c+1 (+8) are this lane's columns
            float kscale[4] = {1.0f, 1.0f, 1.0f, 1.0f}, vexp[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (kE4m3) {
                const unsigned char* me = meta + stage * S::kMeta;
                const uint32_t n = me[S::kByte + lane];
                const uint32_t word = *reinterpret_cast<const volatile uint32_t*>(me + lane * 4);
                const uint32_t byte = n ? (word >> (8 * (n - 1))) & 0xffu : 127u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = 2 * c + (j & 1) + (j >> 1) * 8;
                    kscale[j] = pow2_of_byte(__shfl_sync(0xffffffffu, byte, key));
                    vexp[j] = static_cast<float>(static_cast<int>(__shfl_sync(0xffffffffu, byte, 16 + key)) - 127);
                }
            }
            uint32_t whi[kHalves][2], wlo[kHalves][2];
            float fix[kHalves];
            bool grew = false;
#pragma unroll
            for (int hh = 0; hh < kHalves; ++hh) {
                float x[4], y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool ok = (mask >> (2 * c + (j & 1) + (j >> 1) * 8)) & 1;
                    x[j] = s[j >> 1][hh * 2 + (j & 1)] * qscale[hh];
                    if (kE4m3) x[j] *= kscale[j];
                    x[j] = ok ? x[j] : -INFINITY;
                    y[j] = kE4m3 ? x[j] + vexp[j] : x[j];
                }
                float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float mn = fmaxf(m[hh], top);
                const float ref = mn == -INFINITY ? 0.0f : (kE4m3 ? mn - kShift : mn);
                fix[hh] = mn > m[hh] ? exp2_fast(m[hh] - mn) : 1.0f;
                grew |= mn > m[hh];
                m[hh] = mn;
                float p[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = exp2_fast(y[j] - ref);
                float sum;
                if (kE4m3)
                    sum = (exp2_fast(x[0] - ref) + exp2_fast(x[1] - ref)) + (exp2_fast(x[2] - ref) + exp2_fast(x[3] - ref));
                else
                    sum = (p[0] + p[1]) + (p[2] + p[3]);
                l[hh] = l[hh] * fix[hh] + sum;
                split_pair<kE4m3>(p[0], p[1], whi[hh][0], wlo[hh][0]);
                split_pair<kE4m3>(p[2], p[3], whi[hh][1], wlo[hh][1]);
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int t = 0; t < S::kTiles; ++t) {
                    o[t][0] *= fix[0];
                    o[t][1] *= fix[0];
                    o[t][2] *= fix[kHalves - 1];
                    o[t][3] *= fix[kHalves - 1];
                }
            }

            const uint32_t vt = ring + stage * 2 * S::kTile + S::kTile + lane * S::kValBytes;
#pragma unroll
            for (int u = 0; u < S::kValSegs; ++u) {
                uint32_t v[4][4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t at = vt + (t * S::kValSegs + u) * 32 * S::kValBytes;
                    if (S::kValBytes == 16) {
                        const uint4 w = lds128(at);
                        v[t][0] = w.x;
                        v[t][1] = w.y;
                        v[t][2] = w.z;
                        v[t][3] = w.w;
                    } else {
                        const uint2 w = lds64(at);
                        v[t][0] = w.x;
                        v[t][1] = w.y;
                        v[t][2] = v[t][3] = 0;
                    }
                }
#pragma unroll
                for (int j = 0; j < S::kValElts; ++j) {
                    uint32_t v0, v1;
                    if (kE4m3) {
                        // bytes j of two keys side by side, two j at a time
                        const int w = j >> 2, sel = (j & 2) ? 0x7362 : 0x5140;
                        v0 = f16_of_codes(__byte_perm(v[0][w], v[1][w], sel), j & 1);
                        v1 = f16_of_codes(__byte_perm(v[2][w], v[3][w], sel), j & 1);
                    } else {
                        const int w = j >> 1, sel = (j & 1) ? 0x7632 : 0x5410;
                        v0 = __byte_perm(v[0][w], v[1][w], sel);
                        v1 = __byte_perm(v[2][w], v[3][w], sel);
                    }
                    float(&acc)[4] = o[u * S::kValElts + j];
                    if (kHalves == 1) {
                        mma_16816(acc, whi[0][0], wlo[0][0], whi[0][1], wlo[0][1], v0, v1, kE4m3);
                    } else {
                        mma_16816(acc, whi[0][0], whi[kHalves - 1][0], whi[0][1], whi[kHalves - 1][1], v0, v1, kE4m3);
                        mma_16816(acc, wlo[0][0], wlo[kHalves - 1][0], wlo[0][1], wlo[kHalves - 1][1], v0, v1, kE4m3);
                    }
                }
            }
        }
        __syncwarp();
        if (i + kStages < count) issue(stage);
        copy_commit();
        stage = stage + 1 == kStages ? 0 : stage + 1;

        // ---- the end of an item, or of this block's part of it
        if (cw.g + 1 == cw.n || i + 1 == count) {
            const long long c0 = cw.off / run, c1 = (cw.off + cw.n - 1) / run;   // the item's blocks
            const bool whole = c0 == c1;
            constexpr int kSlot = 16 * D + 32;                                   // floats per part
            float* const slots = reinterpret_cast<float*>(static_cast<char*>(a.ws) + kAttentionCtrlBytes);
            float* const part = slots + (2 * static_cast<size_t>(blockIdx.x) + (c0 == blockIdx.x ? 1 : 0)) * kSlot;
#pragma unroll
            for (int hh = 0; hh < kHalves; ++hh) {
                float sum = l[hh];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (c == 0) s_ml[warp * 16 + hh * 8 + g] = make_float2(m[hh], sum);
            }
            // rows of 8 heads at a time through shared memory: row r of half hh is warp r's (and r + 4's)
#pragma unroll
            for (int hh = 0; hh < kHalves; ++hh) {
                if (hh * 8 >= live_heads) break;
                if (hh > 0) __syncthreads();
                float* dst = s_merge + (warp * 8 + g) * D;
#pragma unroll
                for (int u = 0; u < S::kValSegs; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < S::kValElts; j += 4) {
                            float x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float(&acc)[4] = o[u * S::kValElts + j + k];
                                x[k] = kHalves == 1 ? acc[e] + acc[2 + e] : acc[2 * hh + e];
                            }
                            *reinterpret_cast<float4*>(dst + u * 8 * S::kValElts + (2 * c + e) * S::kValElts + j) =
                                make_float4(x[0], x[1], x[2], x[3]);
                        }
                __syncthreads();
                for (int r = warp; r < 8 && hh * 8 + r < live_heads; r += kWarps) {
                    float M = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w * 16 + hh * 8 + r].x);
                    const float ref = M == -INFINITY ? 0.0f : M;
                    float L = 0.0f, f[kWarps];
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float2 ml = s_ml[w * 16 + hh * 8 + r];
                        f[w] = exp2_fast(ml.x - ref);
                        L += ml.y * f[w];
                    }
                    const int head = head0 + hh * 8 + r;
                    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                    for (int d = 4 * lane; d < D; d += 128) {
                        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                        for (int w = 0; w < kWarps; ++w) {
                            const float4 y = *reinterpret_cast<const float4*>(s_merge + (w * 8 + r) * D + d);
                            x.x += y.x * f[w];
                            x.y += y.y * f[w];
                            x.z += y.z * f[w];
                            x.w += y.w * f[w];
                        }
                        if (whole)
                            *reinterpret_cast<uint2*>(a.out + cw.b * a.out_token_stride + head * a.out_head_stride + d) =
                                make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
                        else
                            *reinterpret_cast<float4*>(part + (hh * 8 + r) * D + d) = x;
                    }
                    if (lane == 0) {
                        if (!whole)
                            *reinterpret_cast<float2*>(part + 16 * D + 2 * (hh * 8 + r)) = make_float2(M, L);
                        else if (a.lse)
                            a.lse[static_cast<long long>(cw.b) * a.n_heads + head] =
                                L == 0.0f ? -INFINITY : ((kE4m3 ? M - kShift : M) + log2f(L)) * kLn2;
                    }
                }
            }
            if (!whole) {
                // the last of the item's blocks joins the parts, in the order of the blocks
                __threadfence();
                __syncthreads();
                const int parts = static_cast<int>(c1 - c0) + 1;
                if (threadIdx.x == 0) {
                    unsigned* counter = reinterpret_cast<unsigned*>(static_cast<char*>(a.ws) + 256) + c0;
                    s_last = atomicInc(counter, parts - 1) == static_cast<unsigned>(parts - 1);   // back to 0 by itself
                    __threadfence();
                }
                __syncthreads();
                if (s_last) {
                    for (int r = warp; r < live_heads; r += kWarps) {
                        const float* base = slots + 2 * static_cast<size_t>(c0) * kSlot;
                        auto slot = [&](int k) { return base + (2 * static_cast<size_t>(k) + (k == 0 ? 1 : 0)) * kSlot; };
                        float M = -INFINITY;
                        for (int k = lane; k < parts; k += 32)
                            M = fmaxf(M, __ldcg(slot(k) + 16 * D + 2 * r));
#pragma unroll
                        for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
                        const float ref = M == -INFINITY ? 0.0f : M;
                        float L = 0.0f;
                        float4 x[(D + 127) / 128];
#pragma unroll
                        for (int e = 0; e < (D + 127) / 128; ++e) x[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                        for (int k = 0; k < parts; ++k) {
                            const float* p = slot(k);
                            const float2 ml = __ldcg(reinterpret_cast<const float2*>(p + 16 * D + 2 * r));
                            const float f = exp2_fast(ml.x - ref);
                            L += ml.y * f;
#pragma unroll
                            for (int e = 0; e < (D + 127) / 128; ++e) {
                                const int d = 4 * lane + 128 * e;
                                if (d < D) {
                                    const float4 y = __ldcg(reinterpret_cast<const float4*>(p + r * D + d));
                                    x[e].x += y.x * f;
                                    x[e].y += y.y * f;
                                    x[e].z += y.z * f;
                                    x[e].w += y.w * f;
                                }
                            }
                        }
                        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                        const int head = head0 + r;
#pragma unroll
                        for (int e = 0; e < (D + 127) / 128; ++e) {
                            const int d = 4 * lane + 128 * e;
                            if (d < D)
                                *reinterpret_cast<uint2*>(a.out + cw.b * a.out_token_stride + head * a.out_head_stride + d) =
                                    make_uint2(pack_bf16x2(x[e].x * inv, x[e].y * inv), pack_bf16x2(x[e].z * inv, x[e].w * inv));
                        }
                        if (lane == 0 && a.lse)
                            a.lse[static_cast<long long>(cw.b) * a.n_heads + head] =
                                L == 0.0f ? -INFINITY : ((kE4m3 ? M - kShift : M) + log2f(L)) * kLn2;
                    }
                }
            }
            __syncthreads();   // the shared rows are free for the next item
        }
        advance<S::kGranule>(a, cw, heads);
    }
}

template <int D, bool kE4m3, int kHeads>
cudaError_t launch_heads(const AttentionArgs& a, cudaStream_t s)
{
    using S = Shape<D, kE4m3>;
    const auto kernel = paged_attention_kernel<D, kE4m3, kHeads>;
    if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), S::kSmem); e != cudaSuccess) return e;
    // one block per SM, fewer when the longest possible batch has fewer granules
    const long long most = static_cast<long long>(a.max_pages) * a.page_size;
    const long long keys = a.window > 0 && a.window < most ? a.window : most;
    const int group = a.n_heads / a.n_kv_heads;
    const long long items = static_cast<long long>(a.B) * a.n_kv_heads * ((group + kHeads - 1) / kHeads);
    const long long granules = (keys + S::kGranule - 1) / S::kGranule;
    long long grid = num_sms() < kAttentionCtas ? num_sms() : kAttentionCtas;
    if (items < grid && granules < grid && items * granules < grid) grid = items * granules;
    kernel<<<static_cast<unsigned>(grid), 32 * S::kWarps, S::kSmem, s>>>(a);
    return cudaGetLastError();
}

template <int D, bool kE4m3>
cudaError_t launch_d(const AttentionArgs& a, cudaStream_t s)
{
    // 8 query heads per block of heads leave the other half of the matrix rows to the weights' low
    // parts; more share one read of the cache between 16 (at D = 256 the registers hold 8)
    if constexpr (D < 256)
        if (a.n_heads / a.n_kv_heads > 8) return launch_heads<D, kE4m3, 16>(a, s);
    return launch_heads<D, kE4m3, 8>(a, s);
}

}  // namespace

size_t paged_attention_ws_bytes(int head_dim)
{
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    return kAttentionCtrlBytes + 2 * static_cast<size_t>(kAttentionCtas) * (16 * head_dim + 32) * 4;
}

cudaError_t launch_paged_attention(const AttentionArgs& a, int head_dim, bool e4m3, cudaStream_t s)
{
    if (a.B <= 0) return cudaSuccess;
    switch (head_dim) {
        case 64: return e4m3 ? launch_d<64, true>(a, s) : launch_d<64, false>(a, s);
        case 128: return e4m3 ? launch_d<128, true>(a, s) : launch_d<128, false>(a, s);
        default: return e4m3 ? launch_d<256, true>(a, s) : launch_d<256, false>(a, s);
    }
}

}  // namespace moe
