// tree_attention.cu -- attention of several new tokens per sequence (a tree of
// drafted tokens, a short run of a prompt) over the paged cache that holds them.
//
// The rows of a key head are its query heads times the sequence's drafted tokens,
// in tiles of 128; a tile with the cache's keys [64 at a time] is a matrix product
// of the shape the tensor cores want, so that is what runs:
//   S[128, 64] = Q K^T       tcgen05.mma, Q and the key tile in shared memory
//   P = 2^(S c - m)          four warps, a row of S a thread (TMEM lane)
//   O[128, D] += P V         tcgen05.mma, P from TMEM (over S), the value tile as
//                            it lies in shared memory: a row is one index of the sum
// P goes in as two bf16 parts, P = hi + lo: one rounding to bf16 would cost as much
// as the output's, and the second product is on units that are idle anyway.  The
// running maximum is raised only when a score passes it by 2^kSlack, so that O is
// rarely touched between products.  Sums are of the unrounded weights, in fp32.
//
// A block is 9 warps: four for the softmax and the output, four that copy, one whose
// first thread issues the products.  A ring of tiles in shared memory takes keys and
// values in turn (cp.async in 16-byte pieces, swizzled as the products read them:
// pages of any size and any strides); e4m3 rows pass through registers and become
// bf16 there, exactly, their power of two included.  D up to 128 leaves room for two
// blocks an SM, which fill each other's gaps.
//
// Work is dealt out as in attention.cu: all (sequence, key head, row tile) items in
// order, each its number of key tiles and a gap long, cut into equal runs for the
// blocks that fit the GPU at once, found on the device from the lengths.  An item cut by
// a run's end leaves parts (O, maximum and sum) in the workspace, joined by a second
// kernel in the order of the blocks.
//
// What a row does not see: keys that no row sees are masked (their value rows are
// written as zeros); in tiles where rows differ the value rows lose their NaN and
// infinities in shared memory, since 0 times them would reach every row, and the rows
// that do see them get them added at the end.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;
constexpr float kNone = -3.402823466e38f;   // a maximum of nothing: finite, so that differences of two are
constexpr int kRowsTile = 128, kKeys = 64;
constexpr int kPanel = kKeys * 128;         // bytes of 64 values of a tile's 64 rows
// Eight warps, so that two blocks an SM leave a thread 128 registers.
constexpr int kSoftmaxWarps = 4, kCopyWarps = 3, kProductWarp = kSoftmaxWarps + kCopyWarps, kThreads = 32 * (kProductWarp + 1);
constexpr int kGap = 4;                     // places of the list that an item's start and end are worth
constexpr int kMaxSms = 152, kMaxBlocks = 2 * kMaxSms;

template <int D, bool kE4m3>
struct Shape {
    static constexpr int kCtas = D <= 128 ? 2 : 1;                        // blocks per SM
    static constexpr int kTile = kPanel * D / 64;                         // bytes of a key or value tile
    static constexpr int kQ = kRowsTile * D * 2;
    static constexpr int kBars = 640;
    static constexpr int kShare = std::min(233472 / kCtas - 1024, 232448);
    // a ring of slots for tiles; e4m3 tiles have half of the room as they come in, in a ring of their own
    static constexpr int kRaw = kE4m3 ? kKeys * D : 0, kRoom = kShare - kBars - kQ;
    static constexpr int kSlots = kE4m3 ? (D == 64 ? 6 : 3) : std::min(kRoom / kTile, 12);
    static constexpr int kRaws = kE4m3 ? (kRoom - kSlots * kTile) / kRaw : 0;
    static constexpr int kSmem = kQ + kSlots * kTile + kRaws * kRaw + kBars;
    static constexpr int kCols = D <= 128 ? 256 : 512;                    // TMEM columns: O, then two tiles of scores
    static constexpr int kPart = kRowsTile * (D + 2);                     // floats of a part
    static_assert(kSlots >= 3 && kSmem <= kShare && D + 2 * kKeys <= kCols, "room");
};

struct Header {   // of the item that begins in a block's run and does not end there
    int b, hk, first_row, rows, last;   // rows of the tile, from first_row on; last: the block that ends it; -1: no such item
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A condition that all lanes of the (converged) warp agree on, in a form that the compiler knows as such.
__device__ __forceinline__ bool uniform(bool x) { return __any_sync(0xffffffffu, x); }

// The warp that issues the products runs as one, and its elected lane issues them under a predicate: in a branch of one
// lane every operand's way into the uniform registers costs some 100 cycles (TAG).
__device__ __forceinline__ uint32_t elected()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// D[tmem] (+)= A[smem] * B[smem]^T, one instruction of K = 16.
__device__ __forceinline__ void mma_if(uint32_t leader, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
// The same with A in TMEM: 8 columns of bf16 pairs.
__device__ __forceinline__ void mma_tmem_a_if(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t leader, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar), "r"(leader)
        : "memory");
}

// A value tile as the MN-major side: 64-value blocks kPanel apart, groups of 8 rows (of the sum's index) 1024 apart.
__device__ __forceinline__ uint64_t sdesc_values(uint32_t saddr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(kPanel >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// A box of the cache's map at (value, token, head, page), counted on `bar`.
__device__ __forceinline__ void copy_box_if(uint32_t leader, uint32_t dst, const CUtensorMap* map, int x, int token, int head, int page,
                                            uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        "\n\t}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(token), "r"(head), "r"(page), "r"(bar), "r"(leader)
        : "memory");
}
// Copies 16 bytes, or writes 16 zeros when !live (src is then not read).
__device__ __forceinline__ void copy_async_or_zeros(uint32_t dst, const void* src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
// One of the barrier's arrivals, once this thread's copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void sts128(uint32_t a, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// Bits 15 and 31: the bf16 values of the pair that are NaN or infinite.
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint32_t without_odd(uint32_t w)
{
    const uint32_t o = odd_bits(w) >> 15;   // 1 in the place of each odd half
    return w & ~(o * 0xffffu);
}
__device__ __forceinline__ uint32_t any_odd(uint4 v) { return odd_bits(v.x) | odd_bits(v.y) | odd_bits(v.z) | odd_bits(v.w); }

// 2^(byte - 127); byte 0 is a subnormal.
__device__ __forceinline__ float pow2_of_byte(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

// Four e4m3 codes times a power of two, as two bf16 pairs: exact.
__device__ __forceinline__ void bf16_of_codes(uint32_t w, float scale, uint32_t& lo, uint32_t& hi)
{
    uint32_t a, b;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a)), y = __half22float2(*reinterpret_cast<const __half2*>(&b));
    lo = pack_bf16x2(x.x * scale, x.y * scale);
    hi = pack_bf16x2(y.x * scale, y.y * scale);
}

__device__ __forceinline__ long long quotient(long long a, long long b)
{
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// ---------------------------------------------------------------- the work list

struct Item {
    int b, h, items;            // sequence; key head * row tiles + row tile; of so many
    int row0, draft;            // its rows of q
    int len, ctx;               // cached tokens; those before the drafted ones (below 0 only with a wrong length)
    int base, n;                // first key of the first tile, tiles
    long long off;              // the item's first place in the list
};

// A sequence's lengths as the checks leave them.
__device__ __forceinline__ void load_seq(const TreeArgs& a, Item& w, bool record)
{
    const int r0 = a.row_start[w.b], r1 = a.row_start[w.b + 1];
    const bool fine = r0 >= 0 && r1 >= r0 && r1 <= a.T && r1 - r0 <= MOE_MAX_DRAFTED;
    w.row0 = r0;
    w.draft = fine ? r1 - r0 : 0;
    // (a tile's keys past the end still have to be int)
    const long long most = min(static_cast<long long>(a.max_pages) * a.page_size, 0x7fff0000LL);
    const int len = a.seq_len[w.b];
    w.len = len < 0 ? 0 : static_cast<int>(min(static_cast<long long>(len), most));
    w.ctx = w.len - w.draft;
    if (record && (!fine || (w.draft > 0 && (w.len != len || w.ctx < 0)))) record_error(a.status, MOE_ERR_INDEX);
    const int first = a.window > 0 && w.ctx > a.window ? w.ctx - a.window : 0;
    w.base = first & ~(kKeys - 1);
    w.n = w.draft > 0 ? static_cast<int>((static_cast<unsigned>(w.len - w.base) + kKeys - 1) / kKeys) : 0;
    w.items = a.n_kv_heads * ((w.draft * (a.n_heads / a.n_kv_heads) + kRowsTile - 1) / kRowsTile);
}
__device__ __forceinline__ int places(const Item& w) { return w.n ? w.n + kGap : 0; }

__device__ __forceinline__ void next_item(const TreeArgs& a, Item& w)
{
    w.off += places(w);
    if (++w.h < w.items) return;
    w.h = 0;
    do {
        if (++w.b >= a.B) {
            w.n = 0;
            return;
        }
        load_seq(a, w, false);
    } while (w.n == 0);
}

// ---------------------------------------------------------------- the main kernel

struct Start {
    Item item;
    int g;   // first tile
};

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads, (Shape<D, kE4m3>::kCtas))
    tree_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const TreeArgs a)
{
    using S = Shape<D, kE4m3>;
    constexpr int kSlots = S::kSlots, kRaws = S::kRaws;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* const s_q = smem;
    unsigned char* const s_ring = smem + S::kQ;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(s_ring + kSlots * S::kTile + kRaws * S::kRaw);
    // A tile's scores are there (two buffers), its weights, its product with the values done; an item's last product
    // done, its output read; its rows of q there, and no longer read.
    constexpr int kFull = 0, kEmpty = kSlots, kSFull = 2 * kSlots, kPFull = kSFull + 2, kODone = kPFull + 2, kOFree = kODone + 1,
                  kQFull = kOFree + 1, kQEmpty = kQFull + 1, kItemDone = kQEmpty + 1, kRawFull = kItemDone + 1, kRawEmpty = kRawFull + (kE4m3 ? kRaws : kCopyWarps),
                  kCount = kRawEmpty + kRaws;
    static_assert(kCount * 8 + static_cast<int>(sizeof(Start)) + 16 * 8 + 16 <= S::kBars, "room for the barriers");
    Start* const s_start = reinterpret_cast<Start*>(bars + kCount);
    long long* const s_scan = reinterpret_cast<long long*>(s_start + 1);
    volatile uint32_t* const s_tmem = reinterpret_cast<volatile uint32_t*>(s_scan + 16);
    volatile int* const s_odd = reinterpret_cast<volatile int*>(s_tmem + 1);   // NaN or infinities were taken from value rows
    auto bar = [&](int i) { return smem_u32(bars + i); };

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // (the same in all lanes)
    const int group = a.n_heads / a.n_kv_heads;

    // ---- the batch's places, and where this block's run begins
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        Item w;
        w.b = b;
        load_seq(a, w, blockIdx.x == 0);
        mine += static_cast<long long>(places(w)) * w.items;
    }
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) s_scan[warp] = incl;
    // drafted tokens without any key (their length is wrong): zeros
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        Item w;
        w.b = b;
        load_seq(a, w, false);
        if (w.draft == 0 || w.n > 0) continue;
        for (int i = threadIdx.x; i < w.draft * a.n_heads * (D / 8); i += kThreads) {
            const int d = i % (D / 8), h = i / (D / 8) % a.n_heads, t = w.row0 + i / (D / 8) / a.n_heads;
            *reinterpret_cast<uint4*>(a.out + t * a.out_token_stride + h * a.out_head_stride + 8 * d) = make_uint4(0, 0, 0, 0);
            if (a.lse && d == 0) a.lse[static_cast<long long>(t) * a.n_heads + h] = -INFINITY;
        }
    }
    __syncthreads();
    long long total = 0, before = incl - mine;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before += s_scan[i];
        total += s_scan[i];
    }
    const long long run = quotient(total + gridDim.x - 1, gridDim.x);    // places per block
    const long long lo = run * blockIdx.x, hi = min(total, lo + run);
    Header* const header = reinterpret_cast<Header*>(static_cast<char*>(a.ws) + kTreeCtrlBytes) + blockIdx.x;
    if (threadIdx.x == 0) header->last = -1;
    if (lo >= hi) return;
    if (mine > 0 && before <= lo && lo < before + mine) {
        Item w;
        w.b = b0;
        w.h = 0;
        w.off = before;
        load_seq(a, w, false);
        while (w.off + static_cast<long long>(places(w)) * w.items <= lo) {
            w.off += static_cast<long long>(places(w)) * w.items;
            ++w.b;
            load_seq(a, w, false);
        }
        w.h = static_cast<int>(quotient(lo - w.off, places(w)));
        w.off += static_cast<long long>(w.h) * places(w);
        int g = static_cast<int>(lo - w.off);
        if (g >= w.n) {
            next_item(a, w);
            g = 0;
        }
        s_start->item = w;
        s_start->g = g;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(bar(kFull + i), 32);
            mbar_init(bar(kEmpty + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kSFull + i), 1);
            mbar_init(bar(kPFull + i), kSoftmaxWarps);
        }
        mbar_init(bar(kODone), 1);
        mbar_init(bar(kOFree), kSoftmaxWarps);
        mbar_init(bar(kQFull), 32 * kCopyWarps);
        mbar_init(bar(kQEmpty), 1);
        mbar_init(bar(kItemDone), 1);
        for (int i = 0; i < (kE4m3 ? kRaws : kCopyWarps); ++i) mbar_init(bar(kRawFull + i), 32);
        for (int i = 0; i < kRaws; ++i) mbar_init(bar(kRawEmpty + i), 1);
        mbar_fence_init();
        *s_odd = 0;
    }
    __syncthreads();
    if (s_start->item.n == 0 || s_start->item.off + s_start->g >= hi) return;   // nothing but gaps
    if (warp == kProductWarp) {
        tmem_alloc(smem_u32(const_cast<uint32_t*>(s_tmem)), S::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    Item it = s_start->item;
    int g0 = s_start->g;          // the segment's tiles: [g0, g1) of the item
    const float c = a.scale == 0.0f ? kLog2e : fabsf(a.scale) * kLog2e;   // (a scale of 0 zeroes q, one below 0 negates it)
    bool ok = true;
    int seg = 0, tiles = 0;       // segments and tiles done

    if (warp >= kSoftmaxWarps && warp < kProductWarp) {
        // ------------------------------------------------------------ copies
        // bf16: a warp takes every third slot's tile as a whole.  e4m3: the first warp copies, the others turn keys and
        // values into bf16.
        const int mine_of = warp - kSoftmaxWarps;
        const uint32_t leader = elected();
        int looked = 0;   // bf16: tiles that this warp has looked at
        if (a.box_rows > 0 && lane == 0) {
            tma_prefetch_desc(&map_k);
            tma_prefetch_desc(&map_v);
        }
        auto page_of = [&](int key) {
            return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(key)) * a.page_mul) >> a.page_shift);
        };
        for (; uniform(it.n > 0 && it.off + g0 < hi && ok); ++seg) {
            const int g1 = static_cast<int>(min(static_cast<long long>(it.n), hi - it.off));
            const int mtiles = it.items / a.n_kv_heads, hk = it.h / mtiles, row_at = (it.h - hk * mtiles) * kRowsTile;
            const int32_t* const table = a.page_table + it.b * a.table_stride;
            const int n0 = 2 * tiles, n_end = 2 * (tiles + g1 - g0);   // the segment's slots
            auto first_key = [&](int n) { return it.base + (g0 + ((n - n0) >> 1)) * kKeys; };
            // pages of this lane's two keys of slot n's tile
            int entry[2];
            auto look_up = [&](int n) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = first_key(n) + 32 * h + lane;
                    entry[h] = n < n_end && key < it.len ? __ldg(table + page_of(key)) : -1;
                }
            };
            // A tile's rows to dst: boxes, or pieces of 16 bytes (zeros where no key is), kRowBytes each; `full` gets 32 arrivals.
            auto copy_tile = [&](int n, const int (&pages)[2], uint32_t dst, uint32_t full) {
                constexpr int kRowBytes = kE4m3 ? D : 2 * D;
                const int k0 = first_key(n), live = min(kKeys, it.len - k0);
                const bool bad = (lane < live && static_cast<unsigned>(pages[0]) >= static_cast<unsigned>(a.n_pages)) ||
                                 (lane + 32 < live && static_cast<unsigned>(pages[1]) >= static_cast<unsigned>(a.n_pages));
                if (a.box_rows > 0 && !uniform(bad)) {
                    const int boxes = (live + a.box_rows - 1) / a.box_rows;
                    if (lane == 0)
                        mbar_arrive_expect_tx(full, static_cast<uint32_t>(boxes * a.box_rows * kRowBytes));
                    else
                        mbar_arrive(full);
                    __syncwarp();
                    for (int j = 0; uniform(j < boxes); ++j) {
                        const int r = j * a.box_rows, key = k0 + r;
                        const int page = __shfl_sync(0xffffffffu, r < 32 ? pages[0] : pages[1], r & 31);
                        const int token = key - page_of(key) * a.page_size;
#pragma unroll
                        for (int x = 0; x < (kE4m3 ? 1 : D / 64); ++x)
                            copy_box_if(leader, dst + x * kPanel + r * (kE4m3 ? D : 128), n & 1 ? &map_v : &map_k, 64 * x, token, hk, page, full);
                    }
                } else {
                    long long place[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = k0 + 32 * h + lane;
                        const bool there = pages[h] >= 0 && pages[h] < a.n_pages;
                        place[h] = there ? pages[h] * a.page_bytes + (key - page_of(key) * a.page_size) * a.token_bytes : -1;
                    }
                    constexpr int kPieces = kRowBytes / 16, kStep = 32 / kPieces, kCount = kKeys * kPieces / 32;
                    const int piece = lane % kPieces, r0 = lane / kPieces;
                    const char* const from = (n & 1 ? a.v : a.k) + hk * a.head_bytes + 16 * piece;
#pragma unroll 8
                    for (int i = 0; i < kCount; ++i) {
                        const int r = i * kStep + r0;
                        const long long p0 = __shfl_sync(0xffffffffu, place[0], r & 31), p1 = __shfl_sync(0xffffffffu, place[1], r & 31);
                        const long long at = r < 32 ? p0 : p1;
                        copy_async_or_zeros(kE4m3 ? dst + r * D + 16 * piece
                                                  : dst + (piece >> 3) * kPanel + r * 128 + (((piece & 7) ^ (r & 7)) << 4),
                                            from + (at < 0 ? 0 : at), at >= 0);
                    }
                    copy_arrive(full);
                }
            };
            // ---- the rows of q, eight at a time; asked for behind the first tile
            auto copy_q = [&]() {
                if (seg > 0) ok = mbar_wait(bar(kQEmpty), (seg - 1) & 1, kSpinBudget);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return false;
                constexpr int kPieces = D / 8;   // 16-byte pieces of a row
                auto at = [&](int r, int piece) {
                    return smem_u32(s_q) + (piece >> 3) * (kRowsTile * 128) + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
                };
#pragma unroll 1
                for (int r1 = 8 * mine_of; r1 < kRowsTile; r1 += 8 * kCopyWarps) {
#pragma unroll
                    for (int i = 0; i < kPieces / 4; ++i) {
                        const int r = r1 + (i * 32 + lane) / kPieces, piece = (i * 32 + lane) % kPieces;
                        const int row = row_at + r, t = row / group;
                        const bool live = t < it.draft && a.scale != 0.0f;
                        copy_async_or_zeros(at(r, piece), a.q + (live ? (it.row0 + t) * a.q_token_stride +
                                                                            (hk * group + (row - t * group)) * a.q_head_stride : 0) + 8 * piece, live);
                    }
                }
                if (a.scale >= 0.0f) {
                    copy_arrive(bar(kQFull));
                } else {
                    copy_wait_all();
#pragma unroll 1
                    for (int r1 = 8 * mine_of; r1 < kRowsTile; r1 += 8 * kCopyWarps)
#pragma unroll
                        for (int i = 0; i < kPieces / 4; ++i) {
                            const uint32_t to = at(r1 + (i * 32 + lane) / kPieces, (i * 32 + lane) % kPieces);
                            const uint4 x = lds128(to);
                            sts128(to, make_uint4(x.x ^ 0x80008000u, x.y ^ 0x80008000u, x.z ^ 0x80008000u, x.w ^ 0x80008000u));
                        }
                    fence_proxy_async_shared();
                    mbar_arrive(bar(kQFull));
                }
                __syncwarp();
                return true;
            };
            // ---- the key and value tiles
            const int odd_from = a.window > 0 ? max(0, it.ctx - a.window + it.draft) : 0;   // below it, and from ctx on, rows differ
            auto mixed = [&](int n) {   // values of a tile where rows differ
                const int k0 = first_key(n);
                return (n & 1) != 0 && (k0 < odd_from || k0 + kKeys > it.ctx);
            };
            auto wait_for = [&](int i, uint32_t parity) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(i), parity, kSpinBudget));
                return ok;
            };
            if constexpr (!kE4m3) {
                int n = n0 + (mine_of + kCopyWarps - n0 % kCopyWarps) % kCopyWarps;
                look_up(n);
                bool q_there = false;
                for (; uniform(n < n_end); n += kCopyWarps) {
                    const int pages[2] = {entry[0], entry[1]};
                    look_up(n + kCopyWarps);
                    if (!wait_for(kEmpty + n % kSlots, ((n / kSlots) & 1) ^ 1)) break;
                    const uint32_t slot = smem_u32(s_ring) + (n % kSlots) * S::kTile;
                    const bool look = uniform(mixed(n));
                    copy_tile(n, pages, slot, look ? bar(kRawFull + mine_of) : bar(kFull + n % kSlots));
                    if (!q_there && !copy_q()) break;
                    q_there = true;
                    if (!look) continue;
                    if (!wait_for(kRawFull + mine_of, looked++ & 1)) break;
                    const int live = min(kKeys, it.len - first_key(n));
                    uint32_t odd = 0;
#pragma unroll 4
                    for (int i = lane; i < S::kTile / 16; i += 32) {   // (rows of 128 bytes: the order within does not matter)
                        const uint32_t at = slot + 16 * i;
                        uint4 x = lds128(at);
                        const bool dead = ((i >> 3) & (kKeys - 1)) >= live;
                        if (dead || any_odd(x)) {
                            odd |= !dead;
                            x = dead ? make_uint4(0, 0, 0, 0) : make_uint4(without_odd(x.x), without_odd(x.y), without_odd(x.z), without_odd(x.w));
                            sts128(at, x);
                        }
                    }
                    if (odd) *s_odd = 1;
                    fence_proxy_async_shared();
                    mbar_arrive(bar(kFull + n % kSlots));
                    __syncwarp();
                }
                if (ok && !q_there && !copy_q()) break;
            } else if (mine_of == 0) {
                int n = n0;
                look_up(n);
                bool q_there = false;
                for (; uniform(n < n_end); n += 2) {   // keys and values of a tile lie in the same pages
                    const int pages[2] = {entry[0], entry[1]};
                    look_up(n + 2);
#pragma unroll 1
                    for (int v = 0; v < 2; ++v) {
                        const int m = n + v;
                        if (!wait_for(kRawEmpty + m % kRaws, ((m / kRaws) & 1) ^ 1)) break;
                        copy_tile(m, pages, smem_u32(s_ring) + kSlots * S::kTile + (m % kRaws) * S::kRaw, bar(kRawFull + m % kRaws));
                    }
                    if (!ok || (!q_there && !copy_q())) break;
                    q_there = true;
                }
            } else {
                if (!copy_q()) break;
                constexpr int kPieces = D / 16, kStep = 32 / kPieces, kCount = kKeys * kPieces / 32;   // pieces of 16 codes
                const int piece = lane % kPieces, r0 = lane / kPieces, v = mine_of - 1;
                const uint8_t* const from_exp = (v ? a.v_exp : a.k_exp) + hk * a.exp_head_stride;
                uint32_t next[2];   // exponent bytes of this lane's two keys
                auto exponents = [&](int n) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = first_key(n) + 32 * h + lane, at = key - page_of(key) * a.page_size;
                        next[h] = entry[h] >= 0 && entry[h] < a.n_pages
                                      ? __ldg(from_exp + entry[h] * a.exp_page_stride + at * a.exp_token_stride) : 127u;
                    }
                };
                look_up(n0 + v);
                exponents(n0 + v);
                look_up(n0 + v + 2);
                for (int n = n0 + v; uniform(n < n_end); n += 2) {
                    const uint32_t exps[2] = {next[0], next[1]};
                    exponents(n + 2);
                    look_up(n + 4);
                    const bool look = uniform(mixed(n));
                    const int live = min(kKeys, it.len - first_key(n));
                    if (!wait_for(kEmpty + n % kSlots, ((n / kSlots) & 1) ^ 1)) break;
                    if (!wait_for(kRawFull + n % kRaws, (n / kRaws) & 1)) break;
                    const uint32_t raw = smem_u32(s_ring) + kSlots * S::kTile + (n % kRaws) * S::kRaw + r0 * D + 16 * piece;
                    const uint32_t slot = smem_u32(s_ring) + (n % kSlots) * S::kTile + (piece >> 2) * kPanel;
                    uint32_t odd = 0;
#pragma unroll 4
                    for (int i = 0; i < kCount; ++i) {
                        const int r = i * kStep + r0;
                        uint4 w = lds128(raw + i * kStep * D);
                        if (r >= live) w = make_uint4(0, 0, 0, 0);
                        const uint32_t e0 = __shfl_sync(0xffffffffu, exps[0], r & 31), e1 = __shfl_sync(0xffffffffu, exps[1], r & 31);
                        const float scale = pow2_of_byte(r < 32 ? e0 : e1);
                        uint4 x, y;
                        bf16_of_codes(w.x, scale, x.x, x.y);
                        bf16_of_codes(w.y, scale, x.z, x.w);
                        bf16_of_codes(w.z, scale, y.x, y.y);
                        bf16_of_codes(w.w, scale, y.z, y.w);
                        if (look && (any_odd(x) | any_odd(y))) {
                            odd = 1;
                            x = make_uint4(without_odd(x.x), without_odd(x.y), without_odd(x.z), without_odd(x.w));
                            y = make_uint4(without_odd(y.x), without_odd(y.y), without_odd(y.z), without_odd(y.w));
                        }
                        const int at = (2 * piece) & 7;
                        sts128(slot + r * 128 + ((at ^ (r & 7)) << 4), x);
                        sts128(slot + r * 128 + (((at + 1) ^ (r & 7)) << 4), y);
                    }
                    if (odd) *s_odd = 1;
                    fence_proxy_async_shared();
                    mbar_arrive(bar(kFull + n % kSlots));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kRawEmpty + n % kRaws));
                    __syncwarp();
                }
            }
            tiles += g1 - g0;
            next_item(a, it);
            g0 = 0;
        }
        copy_wait_all();
        if (!ok) {
            record_error(a.status, MOE_ERR_TIMEOUT);
            for (const long long t0 = clock64(); clock64() - t0 < kSpinBudget / 100;) {   // boxes that nobody waited for land
            }
        }
    } else if (warp == kProductWarp) {
        // ------------------------------------------------------------ products
        {
            const uint32_t leader = elected();
            constexpr uint32_t kIdescS = idesc_bf16_f32(kRowsTile, kKeys), kIdescO = idesc_bf16_f32(kRowsTile, D) | (1u << 16);
            auto wait = [&](int i, uint32_t parity) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(i), parity, kSpinBudget));
                return ok;
            };
            for (; uniform(it.n > 0 && it.off + g0 < hi && ok); ++seg) {
                const int g1 = static_cast<int>(min(static_cast<long long>(it.n), hi - it.off)), count = g1 - g0;
                for (int i = 0; uniform(i <= count && ok); ++i) {
                    const int t = tiles + i, n = 2 * t, u = t - 1, nv = n - 1;   // tile t's scores, tile u's product with the values
                    // The scores take the place of weights that the product two tiles back has read; the slot of its values is
                    // free then, and the keys waited for next may need it.  (Every phase of this barrier is waited for before
                    // the next but one can begin: a wait tells only neighbours apart.)
                    if (uniform(t >= 2 && (i > 0 || seg == 0))) {
                        if (!wait(kODone, t & 1)) break;
                        if (lane == 0) mbar_arrive(bar(kEmpty + (nv - 2) % kSlots));
                        __syncwarp();
                    }
                    if (uniform(i < count) && !wait(kFull + n % kSlots, (n / kSlots) & 1)) break;
                    if (uniform(i == 0) && !wait(kQFull, seg & 1)) break;
                    if (uniform(i > 0) && !wait(kFull + nv % kSlots, (nv / kSlots) & 1)) break;
                    tc_fence_after();
                    fence_proxy_async_shared();   // the copies were written through the generic proxy
                    if (uniform(i < count)) {
                        const uint32_t d = tmem + D + (t & 1) * kKeys, k0 = smem_u32(s_ring) + (n % kSlots) * S::kTile;
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_if(leader, d, sdesc_k_sw128(smem_u32(s_q) + (k >> 2) * (kRowsTile * 128) + (k & 3) * 32),
                                   sdesc_k_sw128(k0 + (k >> 2) * kPanel + (k & 3) * 32), kIdescS, k > 0);
                        commit_if(leader, bar(kSFull + (t & 1)));   // (the keys' slot is handed on by the softmax)
                        if (uniform(i == count - 1)) commit_if(leader, bar(kQEmpty));
                    }
                    if (uniform(i > 0)) {
                        if (!wait(kPFull + (u & 1), (u >> 1) & 1)) break;
                        if (uniform(i == 1 && seg > 0) && !wait(kOFree, (seg - 1) & 1)) break;
                        tc_fence_after();
                        const uint32_t pt = tmem + D + (u & 1) * kKeys, v0 = smem_u32(s_ring) + (nv % kSlots) * S::kTile;
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k) {
                            mma_tmem_a_if(leader, tmem, pt + 8 * k, sdesc_values(v0 + k * 2048), kIdescO, i > 1 || k > 0);
                            mma_tmem_a_if(leader, tmem, pt + kKeys / 2 + 8 * k, sdesc_values(v0 + k * 2048), kIdescO, 1);
                        }
                        commit_if(leader, bar(kODone));
                        if (uniform(i == count)) commit_if(leader, bar(kItemDone));
                    }
                }
                tiles += count;
                next_item(a, it);
                g0 = 0;
            }
            // No arrival on a barrier is under way when the block ends, and no product when TMEM is released.
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(kODone), (tiles - 1) & 1, kSpinBudget));
            if (!ok) {
                if (lane == 0) record_error(a.status, MOE_ERR_TIMEOUT);
                __syncwarp();
                commit_if(leader, bar(kQEmpty));   // counts everything before it
                mbar_wait(bar(kQEmpty), seg & 1, kSpinBudget);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax and output
        const int row = threadIdx.x;
        const uint32_t quarter = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        for (; it.n > 0 && it.off + g0 < hi && ok; ++seg) {
            const int g1 = static_cast<int>(min(static_cast<long long>(it.n), hi - it.off)), count = g1 - g0;
            const int mtiles = it.items / a.n_kv_heads, hk = it.h / mtiles, row_at = (it.h - hk * mtiles) * kRowsTile;
            const int rows = min(kRowsTile, it.draft * group - row_at);
            const bool live = row < rows, idle = warp * 32 >= rows;   // idle: none of the warp's rows is a live one
            const int t_row = (row_at + row) / group, head = hk * group + (row_at + row) - t_row * group;
            // what the row sees: drafted tokens `seen`, context from `from` on
            uint64_t seen = 0;
            int from = 0;
            if (live) {
                seen = a.mask ? a.mask[it.row0 + t_row] : (2ULL << t_row) - 1ULL;
                if (it.draft < 64) seen &= (1ULL << it.draft) - 1ULL;
                if (it.ctx < 0) seen = it.ctx > -64 ? seen & (~0ULL << -it.ctx) : 0ULL;
                if (a.window > 0) {
                    int n = __popcll(seen);
                    for (; n > a.window; --n) seen &= seen - 1;
                    from = max(0, it.ctx - (a.window - n));
                }
            }
            const int32_t* const table = a.page_table + it.b * a.table_stride;
            const int key_lo = it.base + g0 * kKeys, key_hi = min(it.len, it.base + g1 * kKeys);
            // keys of a page out of range are left out: rare, so the segment's part of the table is looked through for one
            bool bad = false;
            if (!idle) {
                for (int pg = key_lo / a.page_size + lane; pg <= (key_hi - 1) / a.page_size; pg += 32) {
                    const int e = __ldg(table + pg);
                    bad = bad || e < 0 || e >= a.n_pages;
                }
                bad = __any_sync(0xffffffffu, bad);
                if (bad && lane == 0) record_error(a.status, MOE_ERR_INDEX);
            }
            const int odd_from = a.window > 0 ? max(0, it.ctx - a.window + it.draft) : 0;
            // bit j: the row sees key k0 + j
            auto sees = [&](int k0) {
                const int lo_bit = min(max(from - k0, 0), 64), hi_bit = min(max(it.ctx - k0, 0), 64);
                uint64_t m = 0;
                if (hi_bit > lo_bit) m = (hi_bit == 64 ? ~0ULL : (1ULL << hi_bit) - 1ULL) & (~0ULL << lo_bit);
                const int shift = k0 - it.ctx;
                if (shift >= 0)
                    m |= shift < 64 ? seen >> shift : 0ULL;
                else
                    m |= shift > -64 ? seen << -shift : 0ULL;
                return m;
            };
            auto resident = [&](int k0) {   // the same of all rows: keys of a page in range
                uint64_t m = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = k0 + 32 * h + lane;
                    const int e = key < it.len ? __ldg(table + key / a.page_size) : -1;
                    m |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, e >= 0 && e < a.n_pages)) << (32 * h);
                }
                return m;
            };
            float m = kNone, l = 0.0f;
            for (int i = 0; i < count; ++i) {
                const int t = tiles + i, k0 = key_lo + i * kKeys;
                if (!__all_sync(0xffffffffu, mbar_wait(bar(kSFull + (t & 1)), (t >> 1) & 1, kSpinBudget))) {
                    ok = false;
                    break;
                }
                if (threadIdx.x == 0) mbar_arrive(bar(kEmpty + (2 * t) % kSlots));   // the keys have been read
                __syncwarp();   // (TMEM is read by whole, converged warps)
                tc_fence_after();
                if (!idle) {
                    const uint32_t at = quarter + D + (t & 1) * kKeys;
                    uint32_t x[2][32];
                    tmem_ld32(at, x[0]);
                    tmem_ld32(at + 32, x[1]);
                    tmem_ld_wait2(x[0], x[1]);
                    if (bad || k0 < odd_from || k0 + kKeys > it.ctx) {
                        uint64_t keep = sees(k0);
                        if (bad) keep &= resident(k0);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t k = static_cast<uint32_t>(keep >> (32 * h));
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!(k >> j & 1u)) x[h][j] = 0xff800000u;
                        }
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 32; ++j) top = fmaxf(top, fmaxf(__uint_as_float(x[0][j]), __uint_as_float(x[1][j])));
                    top *= c;
                    const bool raise = top > m + kSlack;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float to = raise ? top : m, f = raise ? exp2_fast(m - to) : 1.0f;
                        l *= f;
                        m = to;
                        if (i > 0) {
                            if (!__all_sync(0xffffffffu, mbar_wait(bar(kODone), (t - 1) & 1, kSpinBudget))) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll 1
                            for (int d = 0; d < D; d += 32) {
                                uint32_t o[32];
                                tmem_ld32(quarter + d, o);
                                tmem_ld_wait(o);
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st32(quarter + d, o);
                            }
                        }
                    }
                    float sum[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // 32 keys: 16 columns of pairs
                        uint32_t hi_part[16], lo_part[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float p0 = exp2_fast(fmaf(__uint_as_float(x[h][2 * j]), c, -m));
                            const float p1 = exp2_fast(fmaf(__uint_as_float(x[h][2 * j + 1]), c, -m));
                            sum[0] += p0;
                            sum[1] += p1;
                            hi_part[j] = pack_bf16x2(p0, p1);
                            lo_part[j] = pack_bf16x2(p0 - __uint_as_float(hi_part[j] << 16), p1 - __uint_as_float(hi_part[j] & 0xffff0000u));
                        }
                        tmem_st16(at + 16 * h, hi_part);
                        tmem_st16(at + 32 + 16 * h, lo_part);
                    }
                    l += sum[0] + sum[1];
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kPFull + (t & 1)));
            }
            // ---- the segment's output
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(kItemDone), seg & 1, kSpinBudget));
            if (!ok) break;
            tc_fence_after();
            if (!idle) {
                const bool whole = g0 == 0 && g1 == it.n;
                const int slot = 2 * blockIdx.x + (g0 == 0 ? 1 : 0);
                float* const part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + kTreeCtrlBytes + sizeof(Header) * kMaxBlocks) +
                                    static_cast<long long>(slot) * S::kPart;
                const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : NAN);
                const bool odd = *s_odd != 0;
                __nv_bfloat16* const out = a.out + static_cast<long long>(it.row0 + t_row) * a.out_token_stride + static_cast<long long>(head) * a.out_head_stride;
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                    uint32_t o[32];
                    tmem_ld32(quarter + d, o);
                    tmem_ld_wait(o);
                    if (odd) {
                        // value rows of tiles where rows differ have lost their NaN and infinities: to the rows that see them
                        for (int i = 0; i < count; ++i) {
                            const int k0 = key_lo + i * kKeys;
                            if (!(k0 < odd_from || k0 + kKeys > it.ctx)) continue;
                            const uint64_t keep = sees(k0);
                            for (int j = 0; j < kKeys; ++j) {
                                const int key = k0 + j;
                                if (!live || !(keep >> j & 1) || key >= it.len) continue;
                                const int pg = key / a.page_size, e = __ldg(table + pg);
                                if (e < 0 || e >= a.n_pages) continue;
                                const char* const v = a.v + e * a.page_bytes + (key - pg * a.page_size) * a.token_bytes + hk * a.head_bytes;
#pragma unroll
                                for (int u = 0; u < 32; ++u) {
                                    float x = 0.0f;
                                    if (kE4m3) {
                                        const uint8_t code = __ldg(reinterpret_cast<const uint8_t*>(v) + d + u);
                                        if ((code & 0x7f) == 0x7f) x = NAN;
                                    } else {
                                        const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(v) + d + u);
                                        if ((h & 0x7f80u) == 0x7f80u) x = __uint_as_float(h << 16);
                                    }
                                    if (x != 0.0f) o[u] = __float_as_uint(__uint_as_float(o[u]) + x);
                                }
                            }
                        }
                    }
                    if (live && whole) {
#pragma unroll
                        for (int u = 0; u < 32; u += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                w[j] = pack_bf16x2(__uint_as_float(o[u + 2 * j]) * inv, __uint_as_float(o[u + 2 * j + 1]) * inv);
                            *reinterpret_cast<uint4*>(out + d + u) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else if (live) {   // [4 columns][row]: whole lines
#pragma unroll
                        for (int u = 0; u < 32; u += 4)
                            reinterpret_cast<uint4*>(part)[((d + u) >> 2) * kRowsTile + row] = make_uint4(o[u], o[u + 1], o[u + 2], o[u + 3]);
                    }
                    __syncwarp();   // TMEM is read by whole warps
                }
                if (live && whole && a.lse)
                    a.lse[static_cast<long long>(it.row0 + t_row) * a.n_heads + head] = l == 0.0f ? -INFINITY : fmaf(m, kLn2, logf(l));
                if (live && !whole) reinterpret_cast<float2*>(part + kRowsTile * D)[row] = make_float2(m, l);
                if (threadIdx.x == 0 && g0 == 0 && !whole) {
                    Header h;
                    h.b = it.b;
                    h.hk = hk;
                    h.first_row = row_at;
                    h.rows = rows;
                    h.last = static_cast<int>(quotient(it.off + it.n - 1, run));
                    *header = h;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kOFree));
            tiles += count;
            next_item(a, it);
            g0 = 0;
        }
        if (!ok) record_error(a.status, MOE_ERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kProductWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kCols);
    }
}

// ---------------------------------------------------------------- the join

// Block (x, y): the item that begins in block x's run and ends in another's; 32 of its rows, and 32 columns of them.
template <int D>
__global__ void __launch_bounds__(256) tree_attention_join_kernel(const TreeArgs a)
{
    using S = Shape<D, false>;
    const Header h = reinterpret_cast<const Header*>(static_cast<const char*>(a.ws) + kTreeCtrlBytes)[blockIdx.x];
    const int row0 = (blockIdx.y & 3) * 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (h.last < 0 || row0 >= h.rows) return;
    const int row = row0 + lane, col4 = (blockIdx.y >> 2) * 8 + warp;   // four columns
    const int parts = h.last - static_cast<int>(blockIdx.x) + 1;
    const float* const base = reinterpret_cast<const float*>(static_cast<const char*>(a.ws) + kTreeCtrlBytes + sizeof(Header) * kMaxBlocks);
    auto part = [&](int i) { return base + (2LL * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * S::kPart; };
    float m = kNone;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) m = fmaxf(m, reinterpret_cast<const float2*>(part(i) + kRowsTile * D)[row].x);
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float2 ml = reinterpret_cast<const float2*>(part(i) + kRowsTile * D)[row];
        const float4 x = reinterpret_cast<const float4*>(part(i))[col4 * kRowsTile + row];
        const float f = exp2_fast(ml.x - m);
        l = fmaf(ml.y, f, l);
        o.x = fmaf(x.x, f, o.x);
        o.y = fmaf(x.y, f, o.y);
        o.z = fmaf(x.z, f, o.z);
        o.w = fmaf(x.w, f, o.w);
    }
    if (row >= h.rows) return;
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : NAN);
    const int group = a.n_heads / a.n_kv_heads, t = (h.first_row + row) / group, head = h.hk * group + (h.first_row + row) - t * group;
    const long long token = a.row_start[h.b] + t;
    *reinterpret_cast<uint2*>(a.out + token * a.out_token_stride + head * a.out_head_stride + 4 * col4) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (a.lse && col4 == 0) a.lse[token * a.n_heads + head] = l == 0.0f ? -INFINITY : fmaf(m, kLn2, logf(l));
}

template <int D, bool kE4m3>
cudaError_t launch(TreeArgs& a, cudaStream_t s)
{
    using S = Shape<D, kE4m3>;
    const auto kernel = tree_attention_kernel<D, kE4m3>;
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), S::kSmem);
    if (e != cudaSuccess) return e;
    // boxes of as many rows as a page and a tile have in common (the swizzle's pattern is 8 rows high)
    CUtensorMap map_k{}, map_v{};
    int rows = kKeys;
    while (a.page_size % rows != 0) rows /= 2;
    a.box_rows = rows >= 8 && encode_cache_map(&map_k, a.k, kE4m3, D, a.page_size, a.n_kv_heads, a.n_pages, a.token_bytes, a.head_bytes, a.page_bytes, rows) &&
                         encode_cache_map(&map_v, a.v, kE4m3, D, a.page_size, a.n_kv_heads, a.n_pages, a.token_bytes, a.head_bytes, a.page_bytes, rows)
                     ? rows : 0;
    const unsigned grid = static_cast<unsigned>(S::kCtas * std::min(num_sms(), kMaxSms));
    kernel<<<grid, kThreads, S::kSmem, s>>>(map_k, map_v, a);
    tree_attention_join_kernel<D><<<dim3(grid, 4 * D / 32), 256, 0, s>>>(a);
    return cudaGetLastError();
}

template <int D>
size_t ws_bytes()
{
    using S = Shape<D, false>;
    return kTreeCtrlBytes + kMaxBlocks * sizeof(Header) + static_cast<size_t>(S::kCtas) * kMaxSms * 2 * S::kPart * sizeof(float);
}

}  // namespace

size_t tree_attention_ws_bytes(int head_dim)
{
    switch (head_dim) {
        case 64: return ws_bytes<64>();
        case 128: return ws_bytes<128>();
        case 256: return ws_bytes<256>();
        default: return 0;
    }
}

cudaError_t launch_tree_attention(const TreeArgs& args, int head_dim, bool e4m3, cudaStream_t s)
{
    if (args.B <= 0 || args.T <= 0) return cudaSuccess;
    TreeArgs a = args;
    // key / page_size for 0 <= key < 2^31 as a product and a shift: with 2^l the power of two at or above
    // page_size and mul = ceil(2^(31 + l) / page_size), mul * page_size exceeds 2^(31 + l) by less than 2^l
    int l = 0;
    while ((1LL << l) < a.page_size) ++l;
    a.page_shift = 31 + l;
    a.page_mul = static_cast<uint32_t>(((1ULL << (31 + l)) + a.page_size - 1) / a.page_size);
    switch (head_dim) {
        case 64: return e4m3 ? launch<64, true>(a, s) : launch<64, false>(a, s);
        case 128: return e4m3 ? launch<128, true>(a, s) : launch<128, false>(a, s);
        default: return e4m3 ? launch<256, true>(a, s) : launch<256, false>(a, s);
    }
}

}  // namespace moe
