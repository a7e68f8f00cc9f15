// attention.cu -- attention of one new token per sequence over the paged cache.
//
// The cache is read once, so the kernel is a stream of key and value rows
// (2 D elements per key and key head) with little arithmetic on top; its floor
// is the bytes of the live rows at the copy bandwidth.
//
// Work: the live keys of every (sequence, key head, block of query heads) are
// cut into granules of 4 tiles, one per warp.  The granules of the whole batch, in
// that order and with a gap for the end of each item, are dealt out in equal runs
// to the blocks that fit the GPU at once (2 to 4 an SM), whatever the lengths: each
// block finds its run from the lengths alone (a scan over them), so nothing is
// planned on the host and a captured graph follows the lengths.
// A run may end inside an item; such an item's parts (maximum, sum and
// unnormalised output) go to the workspace and the block that finishes last
// joins them, always in the same order.
//
// A warp's tile is 16 keys (32 where a row is at most 128 bytes), copied
// (cp.async) into the warp's own ring of key and value tiles in shared memory,
// which needs no barrier of the block.  All products are m16n8k16 with the cache
// as the 16-row side; the fragments are 16-byte pieces of its rows when the free
// orders are chosen to fit:
//   scores: C[key][head] = K Q^T.  The inner dimension may come in any order if
//   both sides agree: a lane's 16 bytes of a key row are its A fragments of
//   consecutive steps, and the same 16 bytes of a row of Q its B fragments.
//   values: C[d][head] += V^T P.  A lane holds pieces of four keys' rows, which
//   byte permutes pair up over the keys; the order of d is free.  The weights
//   get from the layout of C to that of B by a matrix transpose across the warp.
// The weights go in as the sum of two 16-bit parts (one rounding of them to bf16
// would cost as much as the output's; an f16 one is finer, but not for weights far
// below the largest); with at most 4 query heads the columns 4..7 carry the low
// parts, so both take one product.
//
// The running maximum is raised only when a score passes it by 2^kSlack: the
// weights stay below 2^kSlack, sums are fp32, and the usual tile needs neither
// an exchange between lanes nor a pass over the output registers.
//
// e4m3 rows become f16 in one conversion per two codes (exact), so that path
// multiplies in f16: Q is scaled by a power of two per head, and the value rows'
// exponents enter as 2^(s + e) in the weights, whose running maximum is taken
// over s + e.  The sum of the softmax has a maximum of its own, over s: against
// that of s + e its terms could be anything from 2^-250 to 2^250 (256 sequences
// up to 4096: 179 us with one maximum for both, 181 with two).
//
// Measured (32 query heads on 8, D = 128, 6801 GB/s copied): 64 sequences up to
// 8192, bf16, 1083 MB in 167 us (0.96 of the copy rate); one of 131072, 537 MB in
// 89 us (0.89: the start, and the join of 57 parts for each of 8 key heads); 256 up
// to 4096, e4m3, 64 heads on 8, 1091 MB in 181 us (0.89).  The bf16 kernel waits for
// its copies (issue slots 30% busy).  The e4m3 one has half the bytes per key and the
// same products on top of a conversion per code pair: some 910 instructions per 32
// keys, 55% of its issue slots, and 168 registers leave 12 warps an SM to fill them.
// Of the same batch with a fiftieth of the value rows zeros 207 us (they are looked
// at), with exponents anywhere in 130 powers of two 184.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kAttentionCtas = 4 * 152;   // most blocks of a launch
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;
// e4m3 path: weights are held times 2^6 (at most 2^14), so that f16 keeps those 2^-30 of the maximum's
constexpr float kShift = 6.0f;
// the sum of the softmax stays in fp32, whose range asks for a new maximum less often
constexpr float kSlackSum = 32.0f;
constexpr int kZeroByte = 127;   // the exponent byte of a row of zeros, as the append stores it: an exponent of 0
constexpr float kNone = -3.402823466e38f;   // a maximum of nothing: finite, so that differences of two are

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
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Copies 16 bytes, or writes 16 zeros when !live (src is then not read).
__device__ __forceinline__ void copy_async_or_zeros(uint32_t dst, const void* src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
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

// Four e4m3 codes to two pairs of f16, exactly.
__device__ __forceinline__ void f16_of_codes(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
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

// Transposes an 8 x 8 matrix of 16-bit values held as one pair (row lane / 4, columns 2 (lane % 4) ..) per lane.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
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

// A condition that all lanes of the (converged) warp agree on, in a form that the compiler knows as such: what it cannot
// prove uniform it branches on with reconvergence bookkeeping (256 sequences up to 4096, e4m3: 4% slower without).
__device__ __forceinline__ bool uniform(bool x) { return __any_sync(0xffffffffu, x); }

// *counter == last ? 0 : *counter + 1, and the value before: the block's writes so far (ordered before thread
// 0's arrival by the block's barrier) are visible to whoever reads after a later arrival.
__device__ __forceinline__ unsigned count_arrival(unsigned* counter, unsigned last)
{
    unsigned old;
    asm volatile("atom.inc.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(counter), "r"(last) : "memory");
    return old;
}

// a / b for a >= 0, b > 0: nearly always both fit 32 bits, whose division is far shorter.
__device__ __forceinline__ long long quotient(long long a, long long b)
{
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

template <int D, bool kE4m3, int kHeads>
struct Shape {
    static constexpr int kRow = D * (kE4m3 ? 1 : 2);          // bytes of a row
    static constexpr int kCols = kHeads <= 8 ? 1 : 2;         // column tiles of 8
    static constexpr int kOut = D / 16 * 4 * kCols;           // output registers
    static constexpr int kWarps = 4;
    // blocks per SM, as the registers of outputs and queries allow: 128, 168 or 255 a thread (16 heads of 64, e4m3, whose
    // conversions need more beside them: 64 sequences up to 8192, 128 heads on 8, in 94 us, 132 with three blocks that spill)
    static constexpr int kHeld = kOut + D / 8 * kCols;
    static constexpr int kCtas = kHeld <= 24 ? 4 : (kHeld <= 48 && !(kE4m3 && kCols == 2) ? 3 : 2);
    // 16-key parts of a tile: two where a row is short, so that a pass of the loop does twice the work
    static constexpr int kParts = kRow <= 128 ? 2 : 1;
    static constexpr int kPart = 16 * kRow;                   // bytes of 16 keys
    static constexpr int kTile = kParts * kPart;              // bytes of a warp's key (or value) tile
    static constexpr int kTileKeys = 16 * kParts;
    // tiles whose pages are looked up in advance; the e4m3 loop has no registers for two (186 against 180 us,
    // 256 sequences up to 4096)
    static constexpr int kAhead = kE4m3 ? 1 : 2;
    static constexpr int kGranule = kTileKeys * kWarps;       // keys
    // What an item costs beside its granules (the block's join of its warps, the output or the part): so many places of
    // the list are left empty behind it.  With none the blocks that met the most items set the time (64 + 8 heads of
    // 128, e4m3, 256 sequences up to 4096: 213 us; 1 188, 2 180, 3 182; 512 up to 1024: 154, 131, 125, 129).
    static constexpr int kGap = 2;
    static constexpr int kJoin = D == 64 && kHeads == 16 ? 8 : 4;   // heads that the block joins at a time, as memory allows
    static constexpr int kMerge = kWarps * kJoin * D * 4;
    static constexpr int kStats = kWarps * 16 * (kE4m3 ? 12 : 8);   // bytes: the warps' maxima and sums
    static constexpr int kSlot = 16 * D + 32;                       // floats of a part: outputs, maxima and sums
    // beside a tile: which of its keys are live, and the exponent bytes of its e4m3 keys and values
    static constexpr int kMask = kE4m3 ? 2 * kTileKeys : 0, kMeta = kMask + 4;
    // as many slots (key or value tiles) as the block's share of 228 KB holds beside the join, at most 16
    static constexpr int kShare = 233472 / kCtas - 1024 - 384;
    static constexpr int kRoom = kShare - kMerge - kStats;
    static constexpr int kFit = (2 * kRoom / kWarps - 2 * kMeta) / (2 * kTile + kMeta);
    static constexpr int kSlots = kFit < 16 ? kFit : 16;
    static constexpr int kMetas = (kSlots + 3) / 2;           // tiles begun and not finished
    static constexpr int kRing = kWarps * kSlots * kTile;
    static constexpr int kSmem = kRing + kMerge + kWarps * kMetas * kMeta + kStats;
    static_assert(kSlots >= 3 && kSmem <= kShare && kWarps * kMetas * kMeta % 8 == 0, "the ring");
    static constexpr int kCopyRows = kRow >= 128 ? 4 : 2;     // rows of a part that a lane copies from, 16 bytes of each
    static constexpr int kCopySegs = kRow >= 128 ? kRow / 128 : 1;   // ... per 128-byte segment
    static constexpr int kKeySegs = kRow / 64;                // 16-byte pieces of a key row per lane
    static constexpr int kValBytes = kRow / 8 < 16 ? kRow / 8 : 16;
    static constexpr int kValSegs = kRow / (8 * kValBytes);
    static constexpr int kValElts = kValBytes / (kE4m3 ? 1 : 2);
    static constexpr int kSteps = kE4m3 ? 4 : 2;              // inner steps per 16-byte piece
    static constexpr int kQ = D / 8;                          // B registers of 8 heads
    static constexpr int kTiles = D / 16;                     // output row tiles
};

// One item of the work list while it is walked granule by granule.
struct Walk {
    int b, hk, block;    // sequence, key head, block of query heads
    int len, first, n;   // its live keys [first, len) and its granules (per key head and block)
    int g;               // granule within the item
    long long off;       // the item's first place in the whole list
    // Tiles start at multiples of 16, so that with pages of 16 k tokens the 16 keys of a part lie in one page.
    __device__ __forceinline__ int base() const { return first & ~15; }
};

__device__ __forceinline__ int clamped_len(const AttentionArgs& a, int b, bool record)
{
    // (a tile's keys past the end still have to be int)
    const long long most = min(static_cast<long long>(a.max_pages) * a.page_size, 0x7fff0000LL);
    const int n = a.seq_len[b];
    if (n >= 0 && n <= most) return n;
    if (record) record_error(a.status, MOE_ERR_INDEX);
    return n < 0 ? 0 : static_cast<int>(most);
}

__device__ __forceinline__ int first_key(const AttentionArgs& a, int len)
{
    return a.window > 0 && len > a.window ? len - a.window : 0;
}

template <int kGranule>
__device__ __forceinline__ int granules_of(const AttentionArgs& a, int len)
{
    return static_cast<int>((static_cast<unsigned>(len - (first_key(a, len) & ~15)) + kGranule - 1) / kGranule);
}

template <class S>
__device__ __forceinline__ void load_item(const AttentionArgs& a, Walk& w)
{
    w.len = clamped_len(a, w.b, false);
    w.first = first_key(a, w.len);
    w.n = granules_of<S::kGranule>(a, w.len);
}

// Places of an item of n granules in the list.
template <class S>
__device__ __forceinline__ int places_of(int n)
{
    return n ? n + S::kGap : 0;
}

// To the next item; past the end of the batch the walk stays behind its last one (n = 0).
template <class S>
__device__ __forceinline__ void next_item(const AttentionArgs& a, Walk& w, int blocks)
{
    w.off += places_of<S>(w.n);
    w.g = 0;
    if (++w.block < blocks) return;
    w.block = 0;
    if (++w.hk < a.n_kv_heads) return;
    w.hk = 0;
    do {
        if (++w.b >= a.B) {
            w.n = 0;
            return;
        }
        load_item<S>(a, w);
    } while (w.n == 0);
}

template <int D, bool kE4m3, int kHeads>
__global__ void __launch_bounds__(32 * Shape<D, kE4m3, kHeads>::kWarps, Shape<D, kE4m3, kHeads>::kCtas) paged_attention_kernel(const AttentionArgs a)
{
    using S = Shape<D, kE4m3, kHeads>;
    constexpr int kWarps = S::kWarps, kThreads = 32 * kWarps, kSlots = S::kSlots, kMetas = S::kMetas, kCols = S::kCols;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long s_scan[kWarps];
    __shared__ Walk s_start;
    __shared__ int s_last;
    float* const s_merge = reinterpret_cast<float*>(smem + S::kRing);
    unsigned char* const s_meta = smem + S::kRing + S::kMerge;              // [warp][tile]
    float2* const s_ml = reinterpret_cast<float2*>(s_meta + kWarps * kMetas * S::kMeta);   // [warp][16]
    float* const s_sm = reinterpret_cast<float*>(s_ml + kWarps * 16);                       // [warp][16], e4m3

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int group = a.n_heads / a.n_kv_heads;                 // query heads per key head
    const int blocks = (group + kHeads - 1) / kHeads;           // head blocks per key head
    const int heads = a.n_kv_heads * blocks;                    // items per sequence

    // ---- the batch's places, and where this block's run begins
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b)
        mine += places_of<S>(granules_of<S::kGranule>(a, clamped_len(a, b, blockIdx.x == 0)));
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) s_scan[warp] = incl;
    // sequences without live keys: zeros
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (clamped_len(a, b, false) > 0) continue;
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
    const long long run = quotient(all + gridDim.x - 1, gridDim.x);    // places per block
    const long long lo = run * blockIdx.x, hi = min(all, lo + run);
    if (lo >= hi) return;
    if (mine > 0 && before * heads <= lo && lo < (before + mine) * heads) {
        Walk w{};
        w.b = b0;
        w.off = before * heads;
        load_item<S>(a, w);
        while (w.off + static_cast<long long>(places_of<S>(w.n)) * heads <= lo) {
            w.off += static_cast<long long>(places_of<S>(w.n)) * heads;
            ++w.b;
            load_item<S>(a, w);
        }
        const int h = static_cast<int>(quotient(lo - w.off, places_of<S>(w.n)));
        w.hk = h / blocks;
        w.block = h - w.hk * blocks;
        w.off += static_cast<long long>(h) * places_of<S>(w.n);
        w.g = static_cast<int>(lo - w.off);
        if (w.g >= w.n) next_item<S>(a, w, blocks);
        s_start = w;
    }
    __syncthreads();
    if (s_start.off + s_start.g >= hi) return;   // nothing but gaps

    const uint32_t ring = smem_u32(smem) + warp * kSlots * S::kTile;
    unsigned char* const meta = s_meta + warp * kMetas * S::kMeta;
    Walk iw = s_start, cw = s_start;
    int left = static_cast<int>(hi - cw.off) - cw.g, to_copy = left;   // places from the walks to the end of the run

    // ---- the copying side
    constexpr int kElt = kE4m3 ? 1 : 2;
    // A copy instruction moves four 128-byte lines, eight lanes to a line.  A tile is stored by lines (a
    // 128-byte segment of a row, or two 64-byte rows) whose 16-byte pieces are permuted by an XOR with f(row), so
    // that the copies write whole lines and the fragment reads below hit every bank once: for the keys (8 lanes
    // read 4 pieces of rows 2n, 2n + 1) f flips bit 2 with the row, for the values (2 pieces of rows 2n, 2n + 2,
    // 2n + 4, 2n + 6) bits 1 and 2 with row / 2.
    const int sub = lane >> 3, piece = lane & 7;
    const int row0 = S::kRow >= 128 ? sub : 2 * sub + (piece >> 2);       // the lane's rows: row0, row0 + kStep, ..
    constexpr int kStep = S::kRow >= 128 ? 4 : 8;
    const uint32_t token_bytes = static_cast<uint32_t>(a.token_stride * kElt);
    const uint32_t page_bytes = static_cast<uint32_t>(a.page_stride * kElt);
    const uint32_t to_k = ring + sub * 128 + (S::kRow >= 128 ? piece ^ ((sub & 1) << 2 | sub >> 1) : piece) * 16;
    const uint32_t to_v = ring + sub * 128 + (S::kRow >= 128 ? piece ^ (sub >> 1) << 1 : piece ^ sub << 1) * 16;
    const uint32_t from_k = ring + (S::kRow >= 128 ? g * 128 + (c ^ ((g & 1) << 2 | g >> 1)) * 16 : lane * 16);
    const uint32_t from_v = ring + (S::kRow >= 128 ? c * 256 + (g ^ c << 1) * 16 : c * 128 + ((g >> 1) ^ c << 1) * 16 + (g & 1) * 8);
    // a part's keys lie in one page, and one look-up serves them (64 sequences up to 8192, 167 us, otherwise 172; e4m3 92 and
    // 130)
    const bool one_page = a.page_size % 16 == 0;
    // of the item whose tiles are copied: its table row, this lane's place in a page of its key head (for
    // one_page with the lane's first row), the same in the exponents
    const int32_t* table = nullptr;
    const char *lane_k = nullptr, *lane_v = nullptr;
    long long lane_exp = 0;
    int next_key = 0, ahead_page[S::kAhead][S::kParts];   // of the next tiles of the item
    const char* row_v[S::kParts];     // this lane's first row of the parts whose keys were copied last
    uint32_t rows_live = 0;           // and which of their keys live
    int imeta = 0;
    // e4m3: the exponent bytes of key `lane` of that tile, stored beside it when the next one is issued
    uint32_t exp_k = 0, exp_v = 0;
    unsigned char* exp_to = nullptr;
    auto store_exponents = [&]() {
        if (kE4m3 && exp_to && lane < S::kTileKeys) {
            exp_to[lane] = static_cast<unsigned char>(exp_k);
            exp_to[S::kTileKeys + lane] = static_cast<unsigned char>(exp_v);
        }
        exp_to = nullptr;
    };
    auto start_item = [&]() {
        table = a.page_table + iw.b * a.table_stride;
        long long at = iw.hk * a.head_stride * kElt + (S::kRow >= 128 ? piece : piece & 3) * 16;
        if (one_page) at += row0 * static_cast<long long>(token_bytes);
        lane_k = static_cast<const char*>(a.k) + at;
        lane_v = static_cast<const char*>(a.v) + at;
        if (kE4m3) lane_exp = iw.hk * a.exp_head_stride + (one_page ? (lane & 15) * a.exp_token_stride : 0);
        next_key = iw.base() + iw.g * S::kGranule + warp * S::kTileKeys;
    };
    // The pages of the first keys of a tile's parts (one_page) or of their keys `lane & 15`, asked for one tile
    // before the copies (two within an item, where registers allow).
    auto page_of = [&](int key) {
        return static_cast<uint32_t>((static_cast<uint64_t>(static_cast<uint32_t>(key)) * a.page_mul) >> a.page_shift);
    };
    auto look_up = [&](int tile) {
#pragma unroll
        for (int h = 0; h < S::kParts; ++h) {
            const int key = next_key + tile * S::kGranule + 16 * h + (one_page ? 0 : lane & 15);
            ahead_page[tile][h] = key < iw.len ? __ldg(table + page_of(key)) : -1;
        }
    };
    auto copy_part = [&](uint32_t dst, uint32_t flip, const char* row, uint32_t live, const char* idle) {
        if (uniform(one_page && live == 0xffffu)) {
#pragma unroll
            for (int j = 0; j < S::kCopyRows; ++j) {
                const char* src = row + static_cast<uint64_t>(token_bytes) * (j * kStep);
#pragma unroll
                for (int u = 0; u < S::kCopySegs; ++u)
                    copy_async((S::kRow >= 128 && (j & 1) ? dst ^ flip : dst) + u * 2048 + j * 512, src + u * 128);
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < S::kCopyRows; ++j) {
                const int r = row0 + j * kStep;
                const char* src = one_page ? row + static_cast<uint64_t>(token_bytes) * (j * kStep)
                                           : reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), r)) +
                                                 (S::kRow >= 128 ? piece : piece & 3) * 16;
                const bool ok = (live >> r) & 1;
                src = ok ? src : idle;
#pragma unroll
                for (int u = 0; u < S::kCopySegs; ++u)
                    copy_async_or_zeros((S::kRow >= 128 && (j & 1) ? dst ^ flip : dst) + u * 2048 + j * 512, src + u * 128, ok);
            }
        }
    };
    auto issue_keys = [&](uint32_t slot) {
        // keys [first, len) of the tile
        const int lo_key = max(iw.first - next_key, 0), hi_key = min(max(iw.len - next_key, 0), S::kTileKeys);
        rows_live = lo_key < hi_key ? (0xffffffffu >> (32 - hi_key)) & (0xffffffffu << lo_key) : 0u;
        int next_page[S::kParts], next_at[S::kParts];
#pragma unroll
        for (int h = 0; h < S::kParts; ++h) {
            const int key = next_key + 16 * h + (one_page ? 0 : lane & 15);
            next_page[h] = ahead_page[0][h];
            next_at[h] = key - static_cast<int>(page_of(key) * static_cast<uint32_t>(a.page_size));
            const bool ok_page = static_cast<unsigned>(next_page[h]) < static_cast<unsigned>(a.n_pages);
            const uint32_t part = 0xffffu << (16 * h);
            if (one_page) {
                if (!ok_page) {
                    if ((rows_live & part) && lane == 0) record_error(a.status, MOE_ERR_INDEX);
                    rows_live &= ~part;
                }
            } else {
                const bool mine = (rows_live >> (16 * h + (lane & 15))) & 1;
                if (mine && !ok_page) record_error(a.status, MOE_ERR_INDEX);
                rows_live = (rows_live & ~part) | (__ballot_sync(0xffffffffu, mine && ok_page) & 0xffffu) << (16 * h);
            }
            long long place = static_cast<uint64_t>(static_cast<uint32_t>(next_page[h])) * page_bytes +
                              static_cast<uint64_t>(static_cast<uint32_t>(next_at[h])) * token_bytes;
            if (!one_page) place -= (S::kRow >= 128 ? piece : piece & 3) * 16;   // handed around: without the lane's piece
            row_v[h] = lane_v + place;
            copy_part(to_k + slot + h * S::kPart, 32, lane_k + place, rows_live >> (16 * h) & 0xffffu, static_cast<const char*>(a.k));
        }
        unsigned char* const to = meta + imeta * S::kMeta;
        if (kE4m3) {
            const int h = S::kParts == 2 ? lane >> 4 : 0;
            const int page = S::kParts == 2 && h ? next_page[S::kParts - 1] : next_page[0];
            const int at = S::kParts == 2 && h ? next_at[S::kParts - 1] : next_at[0];
            exp_k = 127;
            exp_v = kZeroByte - 1;
            if (lane < S::kTileKeys && ((rows_live >> lane) & 1)) {
                const long long e = lane_exp + page * a.exp_page_stride + at * a.exp_token_stride;
                exp_k = __ldg(a.k_exp + e);
                exp_v = __ldg(a.v_exp + e);
            }
            exp_to = to;
        }
        if (lane == 0) *reinterpret_cast<uint32_t*>(to + S::kMask) = rows_live;
        imeta = imeta + 1 == kMetas ? 0 : imeta + 1;
        next_key += S::kGranule;
        --to_copy;
        if (uniform(++iw.g == iw.n)) {
            to_copy -= S::kGap;
            next_item<S>(a, iw, blocks);
            if (iw.n > 0) {
                start_item();
                look_up(0);
                if (S::kAhead == 2) look_up(S::kAhead - 1);
            }
        } else {
#pragma unroll
            for (int h = 0; h < S::kParts; ++h)
                if (S::kAhead == 2) ahead_page[0][h] = ahead_page[S::kAhead - 1][h];
            look_up(S::kAhead - 1);
        }
    };
    auto issue_values = [&](uint32_t slot) {
#pragma unroll
        for (int h = 0; h < S::kParts; ++h)
            copy_part(to_v + slot + h * S::kPart, 64, row_v[h], rows_live >> (16 * h) & 0xffffu, static_cast<const char*>(a.v));
    };
    // The run as a sequence of tiles (keys, values, keys, ...): number k goes to slot k % kSlots, issued when number
    // k - kSlots has been used.
    bool keys_issued = false;
    auto issue_next = [&](bool values, uint32_t slot) {
        if (!values) {
            store_exponents();
            keys_issued = uniform(to_copy > 0);
        }
        if (keys_issued) {
            if (values)
                issue_values(slot);
            else
                issue_keys(slot);
        }
        copy_commit();
    };
    constexpr bool kOdd = (kSlots & 1) != 0;

    start_item();
    uint32_t q[kCols][S::kQ];
    // An item's rows of Q as bf16 (e4m3: converted when the item begins): the lane's 16 bytes of each 64 of a key
    // row (e4m3: 32 bytes of 128).
    auto load_q = [&](const Walk& w) {
#pragma unroll
        for (int hh = 0; hh < kCols; ++hh) {
            const int h = kHeads == 4 ? g & 3 : hh * 8 + g;
            const bool ok = h < group - w.block * kHeads;
            const __nv_bfloat16* src = a.q + w.b * a.q_token_stride + (w.hk * group + w.block * kHeads + h) * a.q_head_stride;
#pragma unroll
            for (int u = 0; u < S::kQ / 4; ++u) {
                const uint4 v = ok ? __ldg(reinterpret_cast<const uint4*>(src + (kE4m3 ? (u >> 1) * 64 + c * 16 + (u & 1) * 8 : u * 32 + c * 8)))
                                   : make_uint4(0, 0, 0, 0);
                q[hh][4 * u] = v.x;
                q[hh][4 * u + 1] = v.y;
                q[hh][4 * u + 2] = v.z;
                q[hh][4 * u + 3] = v.w;
            }
        }
    };
    load_q(cw);
    look_up(0);
    if (S::kAhead == 2) look_up(S::kAhead - 1);
#pragma unroll 1
    for (int k = 0; k < kSlots; ++k) issue_next((k & 1) != 0, k * S::kTile);

    // ---- the computing side
    float qscale[kCols][2];           // scores in units of log2: accumulator * qscale (* the key's exponent)
    float o[kCols][S::kTiles][4];
    // of the heads 2c and 2c + 1 of the column tile: the maximum that the weights are taken against, the sum of the
    // softmax, and (e4m3) the maximum that the sum is taken against
    float m[kCols][2], l[kCols][2], sm[kCols][2];
    uint32_t slot = 0;                // byte offset in the ring
    int cmeta = 0;
    for (bool first_tile = true; left > 0; first_tile = false) {
        const int head0 = cw.hk * group + cw.block * kHeads, live_heads = min(kHeads, group - cw.block * kHeads);
        if (uniform(first_tile || cw.g == 0)) {    // a new item
#pragma unroll
            for (int hh = 0; hh < kCols; ++hh) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[hh][e] = sm[hh][e] = kNone;
                    l[hh][e] = 0.0f;
                    qscale[hh][e] = a.scale * kLog2e;
                }
                if (kE4m3) {
                    // bf16 to f16 after a power of two that puts the row's largest value near 2^13: values
                    // down to 2^-27 of it stay exact
                    float top = 0.0f;
#pragma unroll
                    for (int j = 0; j < S::kQ; ++j) {
                        const float x = fabsf(__uint_as_float(q[hh][j] << 16)), y = fabsf(__uint_as_float(q[hh][j] & 0xffff0000u));
                        top = fmaxf(top, x < INFINITY ? x : 0.0f);
                        top = fmaxf(top, y < INFINITY ? y : 0.0f);
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    int e = 13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
                    e = top == 0.0f ? 0 : max(-114, min(100, e));
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                    for (int k = 0; k < 2; ++k) qscale[hh][k] *= __shfl_sync(0xffffffffu, down, (2 * c + k) * 4);
#pragma unroll
                    for (int j = 0; j < S::kQ; ++j)
                        q[hh][j] = pack_f16x2(__uint_as_float(q[hh][j] << 16) * up, __uint_as_float(q[hh][j] & 0xffff0000u) * up);
                }
#pragma unroll
                for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[hh][t][j] = 0.0f;
            }
        }

        // ---- scores of the parts' keys g, g + 8 for the heads 2c, 2c + 1
        copy_wait<kSlots - 1>();
        __syncwarp();
        const unsigned char* const me = meta + cmeta * S::kMeta;
        const uint32_t mask = *reinterpret_cast<const volatile uint32_t*>(me + S::kMask);
        float x[S::kParts][kCols][4];
#pragma unroll
        for (int h = 0; h < S::kParts; ++h) {
#pragma unroll
            for (int hh = 0; hh < kCols; ++hh)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[h][hh][j] = 0.0f;
#pragma unroll
            for (int u = 0; u < S::kKeySegs; ++u) {
                const uint32_t at = (S::kRow >= 128 ? ((from_k + slot) ^ (u & 1) * 64) + (u >> 1) * 2048 : from_k + slot) + h * S::kPart;
                const uint4 v0 = lds128(at), v1 = lds128(at + (S::kRow >= 128 ? 1024 : 512));
                const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                for (int k = 0; k < S::kSteps; ++k) {
                    uint32_t f[4];
                    if (kE4m3) {
                        f16_of_codes(w0[k], f[0], f[2]);
                        f16_of_codes(w1[k], f[1], f[3]);
                    } else {
                        f[0] = w0[2 * (k & 1)];
                        f[1] = w1[2 * (k & 1)];
                        f[2] = w0[2 * (k & 1) + 1];
                        f[3] = w1[2 * (k & 1) + 1];
                    }
                    const int step = (u * S::kSteps + k) * 2;
#pragma unroll
                    for (int hh = 0; hh < kCols; ++hh)
                        mma_16816(x[h][hh], f[0], f[1], f[2], f[3], q[hh][step], q[hh][step + 1], kE4m3);
                }
            }
        }
        __syncwarp();
        issue_next(kOdd, slot);
        slot = slot + S::kTile == kSlots * S::kTile ? 0 : slot + S::kTile;

        // Q of the block's next item arrives while this one ends
        const bool last = uniform(cw.g + 1 == cw.n);
        Walk nw = cw;
        left -= last ? 1 + S::kGap : 1;
        if (last && left > 0) {
            next_item<S>(a, nw, blocks);
            load_q(nw);
        }

        // ---- their weights, scores in log2 units
        float kscale[S::kParts][2], vexp[S::kParts][2];
        if (kE4m3) {
#pragma unroll
            for (int h = 0; h < S::kParts; ++h)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int key = 16 * h + 8 * r + g;
                    kscale[h][r] = pow2_of_byte(*static_cast<const volatile unsigned char*>(me + key));
                    vexp[h][r] = static_cast<float>(static_cast<int>(*static_cast<const volatile unsigned char*>(me + S::kTileKeys + key)) - 127);
                }
        }
        cmeta = cmeta + 1 == kMetas ? 0 : cmeta + 1;
#pragma unroll
        for (int h = 0; h < S::kParts; ++h)
#pragma unroll
            for (int hh = 0; hh < kCols; ++hh)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[h][hh][j] *= qscale[hh][j & 1];
                    if (kE4m3) x[h][hh][j] *= kscale[h][j >> 1];
                }
        if (uniform(mask != (S::kParts == 2 ? 0xffffffffu : 0xffffu))) {
#pragma unroll
            for (int h = 0; h < S::kParts; ++h) {
                const bool ok0 = (mask >> (16 * h + g)) & 1, ok1 = (mask >> (16 * h + 8 + g)) & 1;
#pragma unroll
                for (int hh = 0; hh < kCols; ++hh)
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[h][hh][j] = (j < 2 ? ok0 : ok1) ? x[h][hh][j] : -INFINITY;
            }
        }
        auto y = [&](int h, int hh, int j) { return kE4m3 ? x[h][hh][j] + vexp[h][j >> 1] : x[h][hh][j]; };
        auto top_y = [&](int hh, int e) {
            const float top = fmaxf(y(0, hh, e), y(0, hh, 2 + e));
            return S::kParts == 2 ? fmaxf(top, fmaxf(y(S::kParts - 1, hh, e), y(S::kParts - 1, hh, 2 + e))) : top;
        };
        auto top_x = [&](int hh, int e) {
            const float top = fmaxf(x[0][hh][e], x[0][hh][2 + e]);
            return S::kParts == 2 ? fmaxf(top, fmaxf(x[S::kParts - 1][hh][e], x[S::kParts - 1][hh][2 + e])) : top;
        };
        bool grew = false;   // or (e4m3) a value row may be one of zeros
        if (kE4m3) {
#pragma unroll
            for (int h = 0; h < S::kParts; ++h) grew |= vexp[h][0] == 0.0f || vexp[h][1] == 0.0f;
        }
#pragma unroll
        for (int hh = 0; hh < kCols; ++hh)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                grew |= top_y(hh, e) > m[hh][e] + kSlack;
                if (kE4m3) grew |= top_x(hh, e) > sm[hh][e] + kSlackSum;
            }
        if (__any_sync(0xffffffffu, grew)) {
            if (kE4m3) {
                // A value row of zeros would count as one of values near 448, and beside rows of 1e-6 their weights would lose
                // their bits.  Rows with its exponent are looked at, a lane to a row and each at another piece, until all
                // have shown something else.
                const int at = lane & (S::kTileKeys - 1);
                bool zero = lane < S::kTileKeys && (mask >> at & 1) &&
                            *static_cast<const volatile unsigned char*>(me + S::kTileKeys + at) == kZeroByte;
                if (__any_sync(0xffffffffu, zero)) {
                    copy_wait<kSlots - 1>();
                    __syncwarp();
                    const int r = at & 15;
                    const uint32_t row = ring + slot + (at >> 4) * S::kPart +
                                         (S::kRow >= 128 ? r * 128 : (r >> 1) * 128 + ((r & 1) ^ (r >> 2 & 1)) * 64);
                    constexpr int kLine = S::kRow >= 128 ? 8 : 4;   // pieces of a row side by side
#pragma unroll 1
                    for (int i = 0; i < S::kRow / 16 && __any_sync(0xffffffffu, zero); ++i) {
                        const uint4 v = lds128(row + i / kLine * 2048 + ((i + lane) & (kLine - 1)) * 16);
                        zero = zero && ((v.x | v.y | v.z | v.w) & 0x7f7f7f7fu) == 0;
                    }
                    const uint32_t zeros = __ballot_sync(0xffffffffu, zero);
#pragma unroll
                    for (int h = 0; h < S::kParts; ++h)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            if (zeros >> (16 * h + 8 * k + g) & 1) vexp[h][k] = -INFINITY;
                }
            }
#pragma unroll
            for (int hh = 0; hh < kCols; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // from old to the maximum of it and the tile's: the factor of what was taken against old
                    auto raise = [&](float& old, float top) {
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                        const float mn = fmaxf(old, top), fix = mn > old ? exp2_fast(old - mn) : 1.0f;
                        old = mn;
                        return fix;
                    };
                    const float fix = raise(m[hh][e], top_y(hh, e));
                    l[hh][e] *= kE4m3 ? raise(sm[hh][e], top_x(hh, e)) : fix;
#pragma unroll
                    for (int t = 0; t < S::kTiles; ++t) {
                        o[hh][t][e] *= fix;
                        o[hh][t][2 + e] *= fix;
                    }
                }
        }
        uint32_t whi[S::kParts][kCols][2], wlo[S::kParts][kCols][2];
#pragma unroll
        for (int h = 0; h < S::kParts; ++h)
#pragma unroll
            for (int hh = 0; hh < kCols; ++hh) {
                float p[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = exp2_fast(y(h, hh, j) - (kE4m3 ? m[hh][j & 1] - kShift : m[hh][j & 1]));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (kE4m3)
                        l[hh][e] += exp2_fast(x[h][hh][e] - sm[hh][e]) + exp2_fast(x[h][hh][2 + e] - sm[hh][e]);
                    else
                        l[hh][e] += p[e] + p[2 + e];
                }
                uint32_t h0, l0, h1, l1;
                split_pair<kE4m3>(p[0], p[1], h0, l0);
                split_pair<kE4m3>(p[2], p[3], h1, l1);
                if (kHeads == 4) {
                    whi[h][hh][0] = transpose_8x8(c < 2 ? h0 : l0);
                    whi[h][hh][1] = transpose_8x8(c < 2 ? h1 : l1);
                } else {
                    whi[h][hh][0] = transpose_8x8(h0);
                    whi[h][hh][1] = transpose_8x8(h1);
                    wlo[h][hh][0] = transpose_8x8(l0);
                    wlo[h][hh][1] = transpose_8x8(l1);
                }
            }

        // ---- the weighted values
        copy_wait<kSlots - 1>();
        __syncwarp();
#pragma unroll
        for (int h = 0; h < S::kParts; ++h)
#pragma unroll
            for (int u = 0; u < S::kValSegs; ++u) {
                uint32_t v[4][4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t at = (S::kRow >= 128 ? from_v + slot + u * 2048 + (t & 1) * 128 + (t >> 1) * 1024
                                                        : ((from_v + slot) ^ (t & 1) * 64) + (t >> 1) * 512) + h * S::kPart;
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
                // rows g and g + 8 of an output tile are the dimensions j and j + 1 of the lane's piece
#pragma unroll
                for (int j = 0; j < S::kValElts; j += 2) {
                    uint32_t f[4];
                    if (kE4m3) {
                        // bytes j, j + 1 of two keys side by side
                        const int w = j >> 2, sel = (j & 2) ? 0x7362 : 0x5140;
                        f16_of_codes(__byte_perm(v[0][w], v[1][w], sel), f[0], f[1]);
                        f16_of_codes(__byte_perm(v[2][w], v[3][w], sel), f[2], f[3]);
                    } else {
                        const int w = j >> 1;
                        f[0] = __byte_perm(v[0][w], v[1][w], 0x5410);
                        f[1] = __byte_perm(v[0][w], v[1][w], 0x7632);
                        f[2] = __byte_perm(v[2][w], v[3][w], 0x5410);
                        f[3] = __byte_perm(v[2][w], v[3][w], 0x7632);
                    }
                    const int t = (u * S::kValElts + j) / 2;
#pragma unroll
                    for (int hh = 0; hh < kCols; ++hh) {
                        mma_16816(o[hh][t], f[0], f[1], f[2], f[3], whi[h][hh][0], whi[h][hh][1], kE4m3);
                        if (kHeads != 4) mma_16816(o[hh][t], f[0], f[1], f[2], f[3], wlo[h][hh][0], wlo[h][hh][1], kE4m3);
                    }
                }
            }
        __syncwarp();
        issue_next(!kOdd, slot);
        slot = slot + S::kTile == kSlots * S::kTile ? 0 : slot + S::kTile;

        // ---- the end of an item, or of this block's part of it
        if (last || left <= 0) {
            const bool starts = cw.off >= lo, ends = cw.off + cw.n <= hi, whole = starts && ends;
            constexpr int kSlot = S::kSlot;
            // an output from the sums x of weights and L of the softmax; in e4m3 the one is in units of 2^(M - kShift), the
            // other of 2^Ms (their quotient in two halves: the whole may not fit a float where the output does)
            auto write_row = [&](int head, int d, float4 x, float M, float Ms, float L) {
                const float inv = L == 0.0f ? 0.0f : 1.0f / L, up = kE4m3 ? exp2_fast(0.5f * (M - kShift - Ms)) : 1.0f;
                auto scaled = [&](float v) { return kE4m3 ? v * inv * up * up : v * inv; };
                *reinterpret_cast<uint2*>(a.out + cw.b * a.out_token_stride + head * a.out_head_stride + d) =
                    make_uint2(pack_bf16x2(scaled(x.x), scaled(x.y)), pack_bf16x2(scaled(x.z), scaled(x.w)));
                if (d == 0 && a.lse)
                    a.lse[static_cast<long long>(cw.b) * a.n_heads + head] = L == 0.0f ? -INFINITY : ((kE4m3 ? Ms : M) + log2f(L)) * kLn2;
            };
            // a part, or a group's result; in e4m3 with its softmax's sum as the logarithm, whose rounding is that of a score
            auto write_part = [&](float* to, int r, int d, float4 x, float M, float Ms, float L) {
                *reinterpret_cast<float4*>(to + r * D + d) = x;
                if (d == 0) *reinterpret_cast<float2*>(to + 16 * D + 2 * r) = make_float2(M, !kE4m3 ? L : L == 0.0f ? kNone : Ms + log2f(L));
            };
            float* const slots = reinterpret_cast<float*>(static_cast<char*>(a.ws) + kAttentionCtrlBytes);
            float* const part = slots + (3 * static_cast<size_t>(blockIdx.x) + (starts ? 1 : 0)) * kSlot;
#pragma unroll
            for (int hh = 0; hh < kCols; ++hh) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float sum = l[hh][e];
#pragma unroll
                    for (int off = 4; off <= 16; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                    if (g == 0 && (kHeads != 4 || c < 2)) {
                        s_ml[warp * 16 + hh * 8 + 2 * c + e] = make_float2(m[hh][e], sum);
                        if (kE4m3) s_sm[warp * 16 + hh * 8 + 2 * c + e] = sm[hh][e];
                    }
                }
                if (kHeads == 4) {   // the low parts' columns
#pragma unroll
                    for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[hh][t][j] += __shfl_xor_sync(0xffffffffu, o[hh][t][j], 2);
                }
            }
            // kJoin heads at a time through shared memory
#pragma unroll
            for (int first = 0; first < kHeads; first += S::kJoin) {
                if (first >= live_heads) break;
                if (first > 0) __syncthreads();
                if (S::kJoin == 8 || (c >> 1) == ((first >> 2) & 1)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float* dst = s_merge + (warp * S::kJoin + ((2 * c) & (S::kJoin - 1)) + e) * D + g * S::kValElts;
#pragma unroll
                        for (int u = 0; u < S::kValSegs; ++u)
#pragma unroll
                            for (int j = 0; j < S::kValElts; j += 4) {
                                const int t = (u * S::kValElts + j) / 2;
                                *reinterpret_cast<float4*>(dst + u * 8 * S::kValElts + j) =
                                    make_float4(o[first >> 3][t][e], o[first >> 3][t][2 + e], o[first >> 3][t + 1][e], o[first >> 3][t + 1][2 + e]);
                            }
                    }
                }
                __syncthreads();
                for (int at = threadIdx.x; at < S::kJoin * (D / 4); at += kThreads) {
                    const int r = at / (D / 4), d = at % (D / 4) * 4;
                    if (first + r >= live_heads) break;
                    float M = kNone, Ms = kNone;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        M = fmaxf(M, s_ml[w * 16 + first + r].x);
                        if (kE4m3) Ms = fmaxf(Ms, s_sm[w * 16 + first + r]);
                    }
                    float L = 0.0f;
                    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float2 ml = s_ml[w * 16 + first + r];
                        const float f = exp2_fast(ml.x - M);
                        const float4 y = *reinterpret_cast<const float4*>(s_merge + (w * S::kJoin + r) * D + d);
                        L += ml.y * (kE4m3 ? exp2_fast(s_sm[w * 16 + first + r] - Ms) : f);
                        x.x += y.x * f;
                        x.y += y.y * f;
                        x.z += y.z * f;
                        x.w += y.w * f;
                    }
                    if (whole)
                        write_row(head0 + first + r, d, x, M, Ms, L);
                    else
                        write_part(part, first + r, d, x, M, Ms, L);
                }
            }
            if (!whole) {
                // the last of the item's blocks (first .. first + parts - 1) joins the parts, in their order; when
                // they are many, the last of each group of blocks joins the group's first
                const unsigned first = starts ? blockIdx.x : static_cast<unsigned>(quotient(cw.off, run));
                const int parts = static_cast<int>((ends ? blockIdx.x : static_cast<unsigned>(quotient(cw.off + cw.n - 1, run))) - first) + 1;
                const int mine = static_cast<int>(blockIdx.x - first);
                unsigned* const counters = reinterpret_cast<unsigned*>(static_cast<char*>(a.ws) + 256) + first;
                // whether this block's arrival is the last of `count`, for all its threads
                auto last_of = [&](unsigned* counter, int count) {
                    __syncthreads();
                    if (threadIdx.x == 0) s_last = count_arrival(counter, count - 1) == static_cast<unsigned>(count - 1);
                    __syncthreads();
                    return s_last != 0;
                };
                // Results k0, k0 + stride, .. of the item, `count` of them: to the output, or to k0's group result.
                constexpr int kLoads = S::kCtas == 4 ? 4 : 8;   // results whose loads are in flight, as registers allow
                auto join = [&](int k0, int count, int stride, bool grouped, bool final) {
                    auto slot_of = [&](int i) {
                        const int k = k0 + i * stride;
                        return slots + (3 * static_cast<size_t>(first + k) + (grouped ? 2 : k == 0 ? 1 : 0)) * kSlot;
                    };
                    for (int at = threadIdx.x; at < live_heads * (D / 4); at += kThreads) {
                        const int r = at / (D / 4), d = at % (D / 4) * 4;
                        float M = kNone, Ms = 0.5f * kNone, L = 0.0f;   // (2^(kNone - Ms) is 0)
                        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        for (int i0 = 0; i0 < count; i0 += kLoads) {
                            float2 ml[kLoads];
                            float4 y[kLoads];
#pragma unroll
                            for (int i = 0; i < kLoads; ++i) {
                                const float* p = slot_of(min(i0 + i, count - 1));
                                ml[i] = __ldcg(reinterpret_cast<const float2*>(p + 16 * D + 2 * r));
                                y[i] = __ldcg(reinterpret_cast<const float4*>(p + r * D + d));
                            }
                            float mn = M, sn = Ms;
#pragma unroll
                            for (int i = 0; i < kLoads; ++i) {   // (a repeated one changes nothing)
                                mn = fmaxf(mn, ml[i].x);
                                if (kE4m3) sn = fmaxf(sn, ml[i].y);
                            }
                            const float fix = exp2_fast(M - mn);
                            L *= kE4m3 ? exp2_fast(Ms - sn) : fix;
                            x.x *= fix;
                            x.y *= fix;
                            x.z *= fix;
                            x.w *= fix;
                            M = mn;
                            Ms = sn;
#pragma unroll
                            for (int i = 0; i < kLoads; ++i) {
                                const float w = exp2_fast(ml[i].x - M);
                                if (i0 + i < count) {
                                    L += kE4m3 ? exp2_fast(ml[i].y - Ms) : ml[i].y * w;
                                    x.x += y[i].x * w;
                                    x.y += y[i].y * w;
                                    x.z += y[i].z * w;
                                    x.w += y[i].w * w;
                                }
                            }
                        }
                        if (final)
                            write_row(head0 + r, d, x, M, Ms, L);
                        else
                            write_part(slots + (3 * static_cast<size_t>(first + k0) + 2) * kSlot, r, d, x, M, Ms, L);
                    }
                };
                // groups of about the square root of the parts; none of one block, whose counter and result could meet
                // those of the next item, which starts in this item's last block
                int group = parts;
                if (parts > 16)
                    for (group = 8; group * group < parts || parts % group == 1;) ++group;
                const int groups = (parts + group - 1) / group;
                bool final = groups == 1;
                int k0 = mine / group * group, count = min(group, parts - k0), stride = 1;
                unsigned* counter = final ? counters : counters + kAttentionCtas + k0;
                while (last_of(counter, count)) {
                    join(k0, count, stride, stride > 1, final);
                    if (final) break;
                    final = true;
                    counter = counters;
                    k0 = 0;
                    count = groups;
                    stride = group;
                }
            }
            __syncthreads();   // the shared rows are free for the next item
        }
        if (last)
            cw = nw;
        else
            ++cw.g;
    }
}

template <int D, bool kE4m3, int kHeads>
cudaError_t launch_heads(const AttentionArgs& a, cudaStream_t s)
{
    using S = Shape<D, kE4m3, kHeads>;
    const auto kernel = paged_attention_kernel<D, kE4m3, kHeads>;
    if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), S::kSmem); e != cudaSuccess) return e;
    // every resident block once, fewer when the longest possible batch has fewer granules
    const long long most = static_cast<long long>(a.max_pages) * a.page_size;
    const long long keys = a.window > 0 && a.window < most ? a.window : most;
    const int group = a.n_heads / a.n_kv_heads;
    const long long items = static_cast<long long>(a.B) * a.n_kv_heads * ((group + kHeads - 1) / kHeads);
    const long long granules = (keys + 15 + S::kGranule - 1) / S::kGranule;
    long long grid = std::min(num_sms() * S::kCtas, kAttentionCtas);
    if (items < grid && granules < grid && items * (granules + S::kGap) < grid) grid = items * (granules + S::kGap);
    AttentionArgs b = a;
    // key / page_size for 0 <= key < 2^31 as a product and a shift: with 2^l the power of two at or above
    // page_size and mul = ceil(2^(31 + l) / page_size), mul * page_size exceeds 2^(31 + l) by less than 2^l
    int l = 0;
    while ((1LL << l) < a.page_size) ++l;
    b.page_shift = 31 + l;
    b.page_mul = static_cast<uint32_t>(((1ULL << (31 + l)) + a.page_size - 1) / a.page_size);
    kernel<<<static_cast<unsigned>(grid), 32 * S::kWarps, S::kSmem, s>>>(b);
    return cudaGetLastError();
}

template <int D, bool kE4m3>
cudaError_t launch_d(const AttentionArgs& a, cudaStream_t s)
{
    // Up to 4 query heads per key head take both parts of the weights in one product (64 sequences up to 8192, D = 64,
    // e4m3: 66 us, 68 as 8; bf16 and D = 128 within 1%); at D = 256 the 8-wide form is as fast, and its join is
    // shorter (1 of 777: 9.4 us against 15.4).  More than 8 share one read of the cache between 16 (the same with 128 heads
    // on 8, D = 128: 173 us, 321 as two blocks of 8; e4m3 133 and 174); at D = 256 the registers hold 8.
    const int group = a.n_heads / a.n_kv_heads;
    if constexpr (D < 256) {
        if (group <= 4) return launch_heads<D, kE4m3, 4>(a, s);
        if (group > 8) return launch_heads<D, kE4m3, 16>(a, s);
    }
    return launch_heads<D, kE4m3, 8>(a, s);
}

}  // namespace

size_t paged_attention_ws_bytes(int head_dim)
{
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    return kAttentionCtrlBytes + 3 * static_cast<size_t>(kAttentionCtas) * (16 * head_dim + 32) * 4;
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
