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
// P goes in as two 16-bit parts, P = hi + lo: one rounding to bf16 would cost as much
// as the output's, and the second product is on units that are idle anyway.  The
// running maximum is raised only when a score passes it by 2^kSlack, so that O is
// rarely touched between products.  Sums are of the unrounded weights, in fp32.
//
// A block is 8 warps: four for the softmax and the output, three that copy, one that
// issues the products; two blocks an SM for D up to 128, which fill each other's
// gaps.  Key and value tiles take turns in a ring of slots, each with a pair of
// barriers: full (a box or boxes of TMA landed, or cp.async pieces where a page's
// rows and a tile have no 8 in common) and empty (the product that read it is done).
// Scores have two buffers, so S of a tile is computed while the last one's weights are.
//
// e4m3: keys stay codes and q goes in as two e4m3 rows (kind::f8f6f4), the keys'
// powers of two multiply the scores; value codes become f16 in their slots, times
// 2^(their exponent - the tile's largest), which is exact, and the tile's exponent
// goes into the weights.  Tiles whose exponents lie too far apart for that take a way
// of their own (Apart).
//
// What bounds it: bf16 of 128 and 256 memory (64 sequences of up to 8192, 16 drafted,
// 32 heads on 8: 189 us, 0.87 of the copy rate with the join; 4 x 65536: 179 us,
// 0.90; 256: 347 us, 0.93).  With 64 values a head, and e4m3, a tile has half the bytes and the same
// softmax, and what is left is a block's chain: scores there -> maximum -> weights
// -> products (1100 to 2400 cycles a tile, a good part of it waiting for instructions: the
// roles' loops together are more than the first level of the cache holds, so loops
// are rolled and rare ways are out of line).  Items of at most 64 rows therefore have
// their rows twice in the tile of 128, each copy with half of the tile's keys, joined
// at the end: 4 x 65536 with 16 drafted, 32 heads on 8, e4m3 226 -> 190 us, of 64 bf16 values
// a head 128 -> 116 us (0.69 of the copy rate); 128 sequences of up to 4096, 64 heads on 8,
// e4m3: 242 us, 0.35 of the copy rate.  Of more rows the chain is paid for each tile: 61
// drafted, 64 heads on 8, 4 x 65536: 539 us, 0.39 of its floor, of 64 values a head 390, 0.27.
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
// that do see them get them added at the end.  In other tiles all rows see all keys, and
// outputs that came out as NaN or an infinity are settled at the end (settle_odd).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;
// e4m3: weights are held times 2^6 (at most 2^14), so that f16 keeps those 2^-30 of the maximum's
constexpr float kShift = 6.0f;
// exponents of a tile's rows within this many of the largest: the rows go in relative to it (their bits are f16's then)
constexpr int kNarrow = 14;
constexpr float kNone = -3.402823466e38f;   // a maximum of nothing: finite, so that differences of two are
constexpr int kRowsTile = 128, kKeys = 64;
constexpr int kPanel = kKeys * 128;         // bytes of 64 values of a tile's 64 rows
// Eight warps, so that two blocks an SM leave a thread 128 registers.
constexpr int kSoftmaxWarps = 4, kCopyWarps = 3, kProductWarp = kSoftmaxWarps + kCopyWarps, kThreads = 32 * (kProductWarp + 1);
// Places of the list that an item's start and end are worth (64 sequences of up to 8192: with 2 / 4 / 6 / 8 / 12 places 215 /
// 198 / 198 / 200 / 203 us).
constexpr int kGap = 4;
constexpr int kMaxSms = 152, kMaxBlocks = 2 * kMaxSms;

template <int D, bool kE4m3>
struct Shape {
    static constexpr int kCtas = D <= 128 ? 2 : 1;                        // blocks per SM
    static constexpr int kTile = kPanel * D / 64;                         // bytes of a key or value tile of 16-bit values
    static constexpr int kQ = kRowsTile * D * 2;
    static constexpr int kBars = kE4m3 ? 4096 : 1024;
    // Items of at most 64 rows have them twice in the tile, each half with half of a tile's keys: where the softmax, not the
    // copies, is what takes longest (bf16 of 128 gains nothing: 178 us both ways, and would lose a slot).  The halves are joined
    // through 4 KB of shared memory.
    static constexpr bool kSplit = kE4m3 || D == 64;
    static constexpr int kSwap = kSplit ? 4096 : 0;
    static constexpr int kCut = kE4m3 ? 16 : 32;                          // keys that a turn of the softmax's loops takes (e4m3: 32 lost 5%; bf16, D = 64, without halves: 16 lost 5%)
    static constexpr int kShare = std::min(233472 / kCtas - 1024, 232448), kRoom = kShare - kBars - kSwap - kQ;
    // One ring of slots for tiles; e4m3: one for keys, which stay codes, and one for values, which become f16 in their slots
    // (D = 64: behind the codes).
    static constexpr int kTileK = kE4m3 ? kKeys * D : kTile, kTileV = kE4m3 && D == 64 ? kTile + kKeys * D : kTile;
    static constexpr int kSlotsK = kE4m3 ? (D == 64 ? 6 : 3) : 0, kSlotsV = kE4m3 ? (kRoom - kSlotsK * kTileK) / kTileV : 0;
    static constexpr int kSlots = kE4m3 ? kSlotsK + kSlotsV : std::min(kRoom / kTile, 12);
    static constexpr int kRing = kE4m3 ? kSlotsK * kTileK + kSlotsV * kTileV : kSlots * kTile;
    static constexpr int kSmem = kQ + kRing + kBars + kSwap;
    static constexpr int kCols = D <= 128 ? 256 : 512;                    // TMEM columns: O, then two tiles of scores
    static constexpr int kPart = kRowsTile * (D + 4);                     // floats of a part: O, then maximum, sum and O's maximum
    static_assert(kSlots >= 4 && (!kE4m3 || kSlotsV >= 3) && kSmem <= kShare && D + 2 * kKeys <= kCols, "room");
};

// Of the item that begins in a block's run and does not end there.  Headers go by item while there are no more items than
// blocks, else by block: the join has a few blocks to each.
struct Header {
    int b, hk, first_row, rows;   // rows of the tile, from first_row on
    int first, last;              // the blocks that begin and end it; last -1: no such item
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^x of an exponent that may lie below a normal float's (value rows whose own is near the lowest) is within(x)'s power of two
// times rest_of(x).
constexpr float kLeast = -80.0f;
__device__ __forceinline__ float within(float x) { return x < kLeast ? x + 60.0f : fminf(x, 126.0f); }
__device__ __forceinline__ float rest_of(float x) { return x < kLeast ? 0x1p-60f : 1.0f; }

// Two floats of a packed instruction, each rounded as a single one's.
struct Pair {
    float x, y;
};
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b)
{
    Pair r;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    Pair r;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
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
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// 16 columns, there when it returns.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32])
{
    tmem_ld32(taddr, r);
    tmem_ld_wait(r);
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A condition that all lanes of the (converged) warp agree on, in a form that the compiler knows as such.
__device__ __forceinline__ bool uniform(bool x) { return __any_sync(0xffffffffu, x); }

// The warp that issues the products runs as one, and its elected lane issues them under a predicate: in a branch of one
// lane every operand's way into the uniform registers costs some 100 cycles (4 sequences of 65536, 16 drafted: 222 us so, 195 with a predicate).
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
// The same of e4m3 operands, K = 32.
__device__ __forceinline__ void mma_e4m3_if(uint32_t leader, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
// The same with A in TMEM: 8 columns of pairs.
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
// A K-major operand whose rows are 64 bytes, with the 64-byte swizzle: groups of 8 rows 512 bytes apart.
__device__ __forceinline__ uint64_t sdesc_k_sw64(uint32_t saddr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(512 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(4) << 61;
    return d;
}
// Where byte c of row r of a K-major e4m3 operand of `rows` rows lies: panels of 128 bytes (D = 64: rows of 64), swizzled.
template <int D>
__device__ __forceinline__ uint32_t code_at(uint32_t base, int rows, int r, int c)
{
    if (D == 64) return base + r * 64 + ((((c >> 4) ^ (r >> 1)) & 3) << 4) + (c & 15);
    return base + (c >> 7) * (rows * 128) + r * 128 + ((((c >> 4) ^ r) & 7) << 4) + (c & 15);
}
__device__ __forceinline__ void sts64(uint32_t a, uint2 v)
{
    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(a), "r"(v.x), "r"(v.y) : "memory");
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

// The same of f16 values.
__device__ __forceinline__ uint32_t odd_bits_f16(uint32_t w) { return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u; }
__device__ __forceinline__ uint32_t without_odd_f16(uint32_t w) { return w & ~((odd_bits_f16(w) >> 15) * 0xffffu); }

// Four e4m3 codes as two f16 pairs, times a power of two: exact while the products are f16 values.
__device__ __forceinline__ uint32_t times(uint32_t pair, uint32_t scale)
{
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&pair), *reinterpret_cast<const __half2*>(&scale));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void f16_of_codes(uint32_t w, uint32_t scale, uint32_t& lo, uint32_t& hi)
{
    uint32_t a, b;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
    lo = times(a, scale);
    hi = times(b, scale);
}
// Where byte c of row r of an e4m3 value tile lies in its slot until it is turned into f16: where the second half of each
// 128 f16 values of that row goes (D = 64: behind them), so rows may be read and written one after another.
template <int D>
__device__ __forceinline__ uint32_t raw_at(uint32_t slot, int r, int c)
{
    return D == 64 ? slot + kPanel + r * 64 + c : slot + (c >> 7) * (2 * kPanel) + kPanel + r * 128 + (c & 127);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// e4m3: a row of q goes in times 2^-e as the sum of two e4m3 rows, e the smallest with its largest magnitude (bits `top`,
// sign cleared) at most 448 * 2^e.  A bf16 value is such a sum exactly, down to 2^-10 of the largest; below, the error is
// at most 2^-17 of the largest.
__device__ __forceinline__ int row_exponent(uint32_t top)
{
    const int e = static_cast<int>(top >> 7);
    return e == 255 ? 0 : max(e - 135 + ((top & 127u) > 96u ? 1 : 0), -100);
}
__device__ __forceinline__ uint32_t two_codes(float lo, float hi)
{
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(hi), "f"(lo));
    return two;
}
__device__ __forceinline__ float2 of_two_codes(uint32_t two)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }   // -126 .. 127
__device__ __forceinline__ uint32_t largest(uint32_t top, uint32_t w)
{
    return max(top, max(w & 0x7fffu, w >> 16 & 0x7fffu));
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
    int ordinal;                // among the items
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
    ++w.ordinal;
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

// ---------------------------------------------------------------- e4m3 tiles whose rows' exponents lie far apart
// Each key's score is scaled by its own exponent, its weight by its value row's; the sum of the softmax takes an exponential
// of its own, since against the maximum of score + exponent its terms could be anything.  Rare, so it is kept out of the way of
// the usual path: the scores are read from TMEM again, 16 at a time.
struct Apart {
    uint32_t kb[2], vb[2];   // exponent bytes of the keys `lane` and `lane + 32`
    __device__ __forceinline__ Apart(const TreeArgs& a, const int32_t* table, int len, int k0, int hk, uint32_t info)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int key = k0 + 32 * h + lane, pg = key / a.page_size;
            const int e = key < len ? __ldg(table + pg) : -1;
            const bool there = e >= 0 && e < a.n_pages;
            const long long at = there ? e * a.exp_page_stride + (key - pg * a.page_size) * a.exp_token_stride + hk * a.exp_head_stride : 0;
            kb[h] = there ? __ldg(a.k_exp + at) : 127u;
            vb[h] = there && (info & 256u) ? __ldg(a.v_exp + at) : info & 255u;
        }
    }
    __device__ __forceinline__ float score(uint32_t s, int j, uint64_t keep, float c_row) const
    {
        const float f = fminf(fmaxf(c_row * pow2_of_byte(__shfl_sync(0xffffffffu, j < 32 ? kb[0] : kb[1], j & 31)), 1e-37f), 3e38f);
        return keep >> j & 1 ? __uint_as_float(s) * f : -INFINITY;
    }
    __device__ __forceinline__ float exponent(int j) const
    {
        return static_cast<float>(static_cast<int>(__shfl_sync(0xffffffffu, j < 32 ? vb[0] : vb[1], j & 31)) - 127);
    }
};
// The largest score, and score + exponent, of the keys that the row sees.
__device__ __noinline__ float2 apart_maxima(const TreeArgs& a, uint32_t at, uint64_t keep, const int32_t* table, int len, int k0, int hk, uint32_t info,
                                            float c_row)
{
    const Apart e(a, table, len, k0, hk, info);
    float top = -INFINITY, top_out = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < kKeys; c += 16) {
        uint32_t x[16];
        tmem_ld(at + c, x);
        for (int j = 0; j < 16; ++j) {
            const float v = e.score(x[j], c + j, keep, c_row);
            top = fmaxf(top, v);
            top_out = fmaxf(top_out, v + e.exponent(c + j));
        }
    }
    return make_float2(top, top_out);
}
// Writes the weights over the scores; their sum.
__device__ __noinline__ float apart_weights(const TreeArgs& a, uint32_t at, uint64_t keep, const int32_t* table, int len, int k0, int hk, uint32_t info,
                                            float c_row, float m, float m_out)
{
    const Apart e(a, table, len, k0, hk, info);
    float sum = 0.0f;
#pragma unroll 1
    for (int c = 0; c < kKeys; c += 16) {
        uint32_t x[16], hi_part[8], lo_part[8];
        tmem_ld(at + c, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = c + 2 * j;
            const float s0 = e.score(x[2 * j], k, keep, c_row), s1 = e.score(x[2 * j + 1], k + 1, keep, c_row);
            sum += exp2_fast(s0 - m) + exp2_fast(s1 - m);
            const float p0 = exp2_fast(s0 + (e.exponent(k) + kShift - m_out));
            const float p1 = exp2_fast(s1 + (e.exponent(k + 1) + kShift - m_out));
            hi_part[j] = pack_f16x2(p0, p1);
            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi_part[j]));
            lo_part[j] = pack_f16x2(p0 - back.x, p1 - back.y);
        }
        tmem_st(at + c, hi_part);
        tmem_st(at + c + 8, lo_part);
    }
    return sum;
}

// Bit j: the row that sees the context's keys from `from` on and drafted tokens `seen` sees key k0 + j.
__device__ __forceinline__ uint64_t seen_of(int k0, int from, int ctx, uint64_t seen)
{
    const int lo_bit = min(max(from - k0, 0), 64), hi_bit = min(max(ctx - k0, 0), 64), shift = k0 - ctx;
    uint64_t m = 0;
    if (hi_bit > lo_bit) m = (hi_bit == 64 ? ~0ULL : (1ULL << hi_bit) - 1ULL) & (~0ULL << lo_bit);
    if (shift >= 0)
        m |= shift < 64 ? seen >> shift : 0ULL;
    else
        m |= shift > -64 ? seen << -shift : 0ULL;
    return m;
}
// Value rows of tiles where rows differ have lost their NaN and infinities: to the outputs of the row, or the sums of its
// part, if it sees them.  (Rare, so it is as little code as can be, out of the way.)
template <int D, bool kE4m3>
__device__ __noinline__ void add_odd(const TreeArgs& a, const int32_t* table, __nv_bfloat16* out, float* part, int key_lo, int key_hi, int odd_from,
                                     int ctx, int from, int hk, uint64_t seen)
{
#pragma unroll 1
    for (int key = key_lo; key < key_hi; ++key) {
        const int k0 = key - (key - key_lo) % kKeys;
        if (!(k0 < odd_from || k0 + kKeys > ctx) || !(seen_of(key, from, ctx, seen) & 1)) continue;
        const int pg = key / a.page_size, e = __ldg(table + pg);
        if (e < 0 || e >= a.n_pages) continue;
        const char* const v = a.v + e * a.page_bytes + (key - pg * a.page_size) * a.token_bytes + hk * a.head_bytes;
#pragma unroll 1
        for (int d = 0; d < D; ++d) {
            float x = 0.0f;
            if (kE4m3) {
                if ((__ldg(reinterpret_cast<const uint8_t*>(v) + d) & 0x7f) == 0x7f) x = NAN;
            } else {
                const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(v) + d);
                if ((h & 0x7f80u) == 0x7f80u) x = __uint_as_float(h << 16);
            }
            if (x == 0.0f) continue;
            if (out)
                out[d] = __float2bfloat16(__bfloat162float(out[d]) + x);
            else
                part[(d >> 2) * (4 * kRowsTile) + (d & 3)] += x;
        }
    }
}

// bf16: where a product with the values came out as NaN or an infinity, that of a row is what it sees: the sum of the column's
// values that are either (hi and lo parts of a weight times an infinity make NaN as a rule, a weight too small for a float
// does, and the halves' zeros do).  For a whole warp, a row a lane (`mine`: one with such an output); none: a row with no
// score above -infinity, whose outputs are zeros.
template <int D>
__device__ __noinline__ void settle_odd(const TreeArgs& a, const int32_t* table, __nv_bfloat16* out, float* part, int key_lo, int key_hi, int ctx,
                                        int from, int hk, uint64_t seen, bool mine, bool none)
{
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int d = 0; d < D; ++d) {
        float* const at = part + (d >> 2) * (4 * kRowsTile) + (d & 3);
        const float now = !mine ? 0.0f : (out ? __bfloat162float(out[d]) : *at);
        const bool odd = !(fabsf(now) < INFINITY);
        if (!__any_sync(0xffffffffu, odd)) continue;
        float x = 0.0f;
#pragma unroll 1
        for (int k0 = key_lo; k0 < key_hi && !__all_sync(0xffffffffu, !odd || x != x); k0 += 32) {
            const int key = k0 + lane, pg = key / a.page_size, e = key < key_hi ? __ldg(table + pg) : -1;
            uint32_t h = 0;
            if (e >= 0 && e < a.n_pages)
                h = __ldg(reinterpret_cast<const uint16_t*>(a.v + e * a.page_bytes + (key - pg * a.page_size) * a.token_bytes + hk * a.head_bytes) + d);
            for (uint32_t hits = __ballot_sync(0xffffffffu, (h & 0x7f80u) == 0x7f80u); hits; hits &= hits - 1) {
                const int j = __ffs(hits) - 1;
                const float v = __uint_as_float(__shfl_sync(0xffffffffu, h, j) << 16);
                if (seen_of(k0 + j, from, ctx, seen) & 1) x += v;
            }
        }
        if (!odd || (x == 0.0f && !none)) continue;
        if (none) x = 0.0f;
        if (out)
            out[d] = __float2bfloat16(x);
        else
            *at = x;
    }
}

// A wait has run out: the items of the block's run that have no header yet get one that the join passes over, since what the
// workspace held before is no header.  (From the item at hand on; g0 > 0: it began in another block.)
__device__ __noinline__ void give_up(const TreeArgs& a, Header* headers, Item w, int g0, long long hi)
{
    for (; w.n > 0 && w.off + g0 < hi; next_item(a, w), g0 = 0)
        if (g0 == 0) headers[w.ordinal].last = -1;
}

// ---------------------------------------------------------------- the main kernel

struct Start {
    Item item;
    int g;   // first tile
};

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads, (Shape<D, kE4m3>::kCtas))
    tree_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                          const __grid_constant__ TreeArgs a)
{
    using S = Shape<D, kE4m3>;
    constexpr int kSlots = S::kSlots;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* const s_q = smem;
    unsigned char* const s_ring = smem + S::kQ;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(s_ring + S::kRing);
    // A tile's scores are there (two buffers), its weights, its product with the values done; an item's last product
    // done, its output read; its rows of q there, and no longer read.  e4m3: a slot's codes there; bf16: a tile that the
    // warp which copies it looks at.  One half's sums there, and read, for each of two pairs of warps.
    constexpr int kInfos = 8;
    constexpr int kFull = 0, kEmpty = kSlots, kSFull = 2 * kSlots, kPFull = kSFull + 2, kODone = kPFull + 2, kOFree = kODone + 1,
                  kQFull = kOFree + 1, kQEmpty = kQFull + 1, kItemDone = kQEmpty + 1, kRawFull = kItemDone + 1, kSwapFull = kRawFull + (kE4m3 ? S::kSlotsV : kCopyWarps), kSwapEmpty = kSwapFull + 2, kCount = kSwapFull + (S::kSplit ? 4 : 0);
    static_assert(kCount * 8 + static_cast<int>(sizeof(Start)) + 16 * 8 + 16 + (kE4m3 ? kInfos * (4 + 4 * kKeys) + S::kSlotsV * kKeys + 4 * kRowsTile : 0) <= S::kBars, "room for the barriers");
    Start* const s_start = reinterpret_cast<Start*>(bars + kCount);
    long long* const s_scan = reinterpret_cast<long long*>(s_start + 1);
    volatile uint32_t* const s_tmem = reinterpret_cast<volatile uint32_t*>(s_scan + 16);
    volatile int* const s_odd = reinterpret_cast<volatile int*>(s_tmem + 1);   // NaN or infinities were taken from value rows
    // e4m3: of tile t at t % kInfos: its values' exponent byte, bit 8: each row's own; and 2^exponent of each key.  (The tile
    // that is copied is at most 7 ahead of the softmax.)  Of the slots' value rows the exponent bytes.
    float* const s_kf = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(const_cast<uint32_t*>(s_tmem) + 2) + 15) & ~static_cast<uintptr_t>(15));
    volatile uint32_t* const s_info = reinterpret_cast<volatile uint32_t*>(s_kf + kInfos * kKeys);
    volatile uint8_t* const s_exp = reinterpret_cast<volatile uint8_t*>(const_cast<uint32_t*>(s_info) + kInfos);
    // Exponents of the rows of q, of item i at i % 4.  (Those of item i + 4 are written when the scores of item i + 3 are
    // done; the weights of item i are done then, so they have been read.)
    volatile int8_t* const s_qe = reinterpret_cast<volatile int8_t*>(s_exp + (kE4m3 ? S::kSlotsV * kKeys : 0));
    auto bar = [&](int i) { return smem_u32(bars + i); };
    // Tiles are numbered through all of the block's items, keys of tile t as 2 t and values as 2 t + 1: their slot (a barrier's
    // index too), how often it has gone round, and where it is.
    struct Slot {
        int index;
        uint32_t turn, at;
    };
    auto slot_of = [&](int n) {
        Slot o;
        const uint32_t ring = smem_u32(s_ring);
        if constexpr (!kE4m3) {
            o.index = n % kSlots;
            o.turn = static_cast<uint32_t>(n / kSlots) & 1;
            o.at = ring + o.index * S::kTile;
        } else {
            const int t = n >> 1, k = t % S::kSlotsK, v = t % S::kSlotsV;
            o.index = n & 1 ? S::kSlotsK + v : k;
            o.turn = static_cast<uint32_t>(n & 1 ? t / S::kSlotsV : t / S::kSlotsK) & 1;
            o.at = n & 1 ? ring + S::kSlotsK * S::kTileK + v * S::kTileV : ring + k * S::kTileK;
        }
        return o;
    };

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // (the same in all lanes)
    const int group = a.n_heads / a.n_kv_heads;

    let_next_start();
    // ---- the batch's places, and where this block's run begins
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    int mine_items = 0;
    for (int b = b0; b < b1; ++b) {
        Item w;
        w.b = b;
        load_seq(a, w, blockIdx.x == 0);
        mine += static_cast<long long>(places(w)) * w.items;
        mine_items += w.n ? w.items : 0;
    }
    long long incl = mine;
    int incl_items = mine_items;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, off);
        const int i = __shfl_up_sync(0xffffffffu, incl_items, off);
        if (lane >= off) {
            incl += o;
            incl_items += i;
        }
    }
    if (lane == 31) {
        s_scan[warp] = incl;
        s_scan[kThreads / 32 + warp] = incl_items;
    }
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
    int items = 0, before_items = incl_items - mine_items;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) {
            before += s_scan[i];
            before_items += static_cast<int>(s_scan[kThreads / 32 + i]);
        }
        total += s_scan[i];
        items += static_cast<int>(s_scan[kThreads / 32 + i]);
    }
    const long long run = quotient(total + gridDim.x - 1, gridDim.x);    // places per block
    const long long lo = run * blockIdx.x, hi = min(total, lo + run);
    Header* const headers = reinterpret_cast<Header*>(static_cast<char*>(a.ws) + kTreeCtrlBytes);
    // Sequences that share rows, in a row_start that falls and rises again, may have more items than the launch made room for.
    // A block then has the items that begin in its run as a whole, and no header says anything.
    const bool uncut = a.by_item > 0 && items > a.by_item;
    if (a.by_item == 0) {
        if (threadIdx.x == 0) headers[blockIdx.x].last = -1;
    } else if (blockIdx.x == 0) {
        for (int i = (uncut ? 0 : items) + static_cast<int>(threadIdx.x); i < a.by_item; i += kThreads) headers[i].last = -1;
    }
    if (lo >= hi) return;
    if (mine > 0 && before <= lo && lo < before + mine) {
        Item w;
        w.b = b0;
        w.h = 0;
        w.off = before;
        w.ordinal = before_items;
        load_seq(a, w, false);
        while (w.off + static_cast<long long>(places(w)) * w.items <= lo) {
            w.off += static_cast<long long>(places(w)) * w.items;
            w.ordinal += w.n ? w.items : 0;
            ++w.b;
            load_seq(a, w, false);
        }
        w.h = static_cast<int>(quotient(lo - w.off, places(w)));
        w.ordinal += w.h;
        w.off += static_cast<long long>(w.h) * places(w);
        int g = static_cast<int>(lo - w.off);
        if (g >= w.n || (uncut && g > 0)) {
            next_item(a, w);
            g = 0;
        }
        s_start->item = w;
        s_start->g = g;
    }
    static_assert(kCount <= kThreads, "a thread to each barrier");
    if (threadIdx.x < kCount) {
        const int i = threadIdx.x, copies = a.box_rows > 0 ? 1 : 32;   // one arrival by boxes, else each lane's
        int count = 1;
        if (i < kEmpty) count = kE4m3 && i >= S::kSlotsK ? kCopyWarps - 1 : copies;   // (e4m3 values: the warps that turn them into f16)
        if (i >= kRawFull && i < kSwapFull) count = copies;
        if ((i >= kPFull && i < kODone) || i == kOFree) count = kSoftmaxWarps;
        if (i == kQFull) count = 32 * (kE4m3 ? kCopyWarps - 1 : kCopyWarps);
        mbar_init(bar(i), count);
        mbar_fence_init();
    }
    if (threadIdx.x == 0) *s_odd = 0;
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
    auto end_of = [&](const Item& w) { return uncut ? w.n : static_cast<int>(min(static_cast<long long>(w.n), hi - w.off)); };

    if (warp >= kSoftmaxWarps && warp < kProductWarp) {
        // ------------------------------------------------------------ copies
        // bf16: a warp takes every third slot's tile as a whole.  e4m3: the first warp copies, the others turn rows of q into two
        // of e4m3 and values into f16.
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
            const int g1 = end_of(it);
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
            // Slot n's rows to its place (e4m3: and those of the next slot, the same keys' values, to theirs): boxes, or pieces of
            // 16 bytes (zeros where no key is).  Counted on full[0] (and full[1]).
            constexpr int kSides = kE4m3 ? 2 : 1;
            auto copy_tile = [&](int n, const int (&pages)[2], const uint32_t (&dst)[kSides], const uint32_t (&full)[kSides]) {
                constexpr int kRowBytes = kE4m3 ? D : 2 * D;
                const int k0 = first_key(n), live = min(kKeys, it.len - k0);
                const bool bad = (lane < live && static_cast<unsigned>(pages[0]) >= static_cast<unsigned>(a.n_pages)) ||
                                 (lane + 32 < live && static_cast<unsigned>(pages[1]) >= static_cast<unsigned>(a.n_pages));
                if (a.box_rows > 0 && !uniform(bad)) {
                    const uint32_t bytes = static_cast<uint32_t>((live + a.box_rows - 1) / a.box_rows * a.box_rows * kRowBytes);
                    if (lane == 0)
#pragma unroll
                        for (int v = 0; v < kSides; ++v) mbar_arrive_expect_tx(full[v], bytes);
                    // lane j: where box j begins (at most eight of them)
                    const int first = min(lane * a.box_rows, kKeys - 1), at_page = __shfl_sync(0xffffffffu, pages[0], first & 31),
                              at_page1 = __shfl_sync(0xffffffffu, pages[1], first & 31);
                    const int box_page = first < 32 ? at_page : at_page1, box_token = k0 + first - page_of(k0 + first) * a.page_size;
#pragma unroll 1
                    for (int j = 0, r = 0; uniform(r < live); ++j, r += a.box_rows) {
                        const int page = __shfl_sync(0xffffffffu, box_page, j), token = __shfl_sync(0xffffffffu, box_token, j);
#pragma unroll
                        for (int v = 0; v < kSides; ++v)
#pragma unroll
                            for (int x = 0; x < (kE4m3 ? (D + 127) / 128 : D / 64); ++x)
                                copy_box_if(leader, kE4m3 && v == 1 ? raw_at<D>(dst[v], r, 128 * x)
                                                                    : dst[v] + x * kPanel + r * (kE4m3 && D == 64 ? 64 : 128),
                                            (kE4m3 ? v : n & 1) ? &map_v : &map_k, (kE4m3 ? 128 : 64) * x, token, hk, page, full[v]);
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
#pragma unroll 1
                    for (int v = 0; v < kSides; ++v) {
                        const char* const from = ((kE4m3 ? v : n & 1) ? a.v : a.k) + hk * a.head_bytes + 16 * piece;
                        const uint32_t to = kE4m3 && v ? dst[kSides - 1] : dst[0];
#pragma unroll 4
                        for (int i = 0; i < kCount; ++i) {
                            const int r = i * kStep + r0;
                            const long long p0 = __shfl_sync(0xffffffffu, place[0], r & 31), p1 = __shfl_sync(0xffffffffu, place[1], r & 31);
                            const long long at = r < 32 ? p0 : p1;
                            copy_async_or_zeros(kE4m3 ? (v ? raw_at<D>(to, r, 16 * piece) : code_at<D>(to, kKeys, r, 16 * piece))
                                                      : to + (piece >> 3) * kPanel + r * 128 + (((piece & 7) ^ (r & 7)) << 4),
                                                from + (at < 0 ? 0 : at), at >= 0);
                        }
                    }
                    if (a.box_rows > 0) {   // (a page out of range: the barriers count one arrival)
                        copy_wait_all();
                        fence_proxy_async_shared();
                        __syncwarp();
                    }
                    if (a.box_rows == 0 || lane == 0)
#pragma unroll
                        for (int v = 0; v < kSides; ++v) copy_arrive(full[v]);
                    __syncwarp();
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
                const int rows = a.scale != 0.0f ? it.draft * group - row_at : 0;   // live ones
                const bool twice = S::kSplit && it.draft * group - row_at <= kRowsTile / 2;
                const int distinct = twice ? kRowsTile / 2 : kRowsTile;
                if constexpr (kE4m3) {
                    // Two e4m3 rows for each, one tile behind the other.  (One piece a turn: the code is run once an item, so what it
                    // costs is to fetch it.)
                    constexpr int kRows = 32 / kPieces, kStep = kRows * (kCopyWarps - 1);   // rows of a warp at a time
                    const int piece = lane % kPieces;
                    auto fetch = [&](int r) {
                        if (r >= rows || r >= kRowsTile) return make_uint4(0, 0, 0, 0);
                        const int t = a.tokens_of(row_at + r);
                        return __ldg(reinterpret_cast<const uint4*>(a.q + (it.row0 + t) * a.q_token_stride +
                                                                    (hk * group + (row_at + r - t * group)) * a.q_head_stride + 8 * piece));
                    };
                    int r = kRows * (mine_of - 1) + lane / kPieces;
                    uint4 next = fetch(r), after = fetch(r + kStep);
#pragma unroll 1
                    for (; uniform(r - lane / kPieces < distinct); r += kStep) {
                        const uint4 x = next;
                        next = after;
                        after = fetch(r + 2 * kStep);
                        uint32_t top = largest(largest(largest(largest(0, x.x), x.y), x.z), x.w);
#pragma unroll
                        for (int off = kPieces / 2; off >= 1; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
                        const int e = row_exponent(top);
                        // (a row with a NaN or an infinity is NaN)
                        const float f = top >> 7 == 255u ? NAN : (a.scale < 0.0f ? -1.0f : 1.0f) * pow2(-e);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                        uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float v0 = __uint_as_float(w[j] << 16) * f, v1 = __uint_as_float(w[j] & 0xffff0000u) * f;
                            const uint32_t two = two_codes(v0, v1);
                            const float2 back = of_two_codes(two);
                            hi[j >> 1] |= two << (16 * (j & 1));
                            lo[j >> 1] |= two_codes(v0 - back.x, v1 - back.y) << (16 * (j & 1));
                        }
                        if (r < distinct) {
                            sts64(code_at<D>(smem_u32(s_q), kRowsTile, r, 8 * piece), make_uint2(hi[0], hi[1]));
                            sts64(code_at<D>(smem_u32(s_q) + kRowsTile * D, kRowsTile, r, 8 * piece), make_uint2(lo[0], lo[1]));
                            if (twice) {
                                sts64(code_at<D>(smem_u32(s_q), kRowsTile, r + distinct, 8 * piece), make_uint2(hi[0], hi[1]));
                                sts64(code_at<D>(smem_u32(s_q) + kRowsTile * D, kRowsTile, r + distinct, 8 * piece), make_uint2(lo[0], lo[1]));
                            }
                            if (piece == 0) s_qe[(seg & 3) * kRowsTile + r] = static_cast<int8_t>(e);
                        }
                    }
                    fence_proxy_async_shared();
                    mbar_arrive(bar(kQFull));
                    __syncwarp();
                    return true;
                } else {
#pragma unroll 1
                    for (int r1 = 8 * mine_of; r1 < kRowsTile; r1 += 8 * kCopyWarps) {
                        // lane j: row r1 + j % 8
                        const int first = r1 & (distinct - 1), mine = first + (lane & 7), t = a.tokens_of(row_at + mine);
                        const long long place = mine < rows ? (it.row0 + t) * a.q_token_stride +
                                                                  (hk * group + (row_at + mine - t * group)) * a.q_head_stride : 0;
#pragma unroll
                        for (int i = 0; i < kPieces / 4; ++i) {
                            const int r = (i * 32 + lane) / kPieces, piece = (i * 32 + lane) % kPieces;
                            const long long from = __shfl_sync(0xffffffffu, place, r);
                            copy_async_or_zeros(at(r1 + r, piece), a.q + from + 8 * piece, first + r < rows);
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
                }
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
                bool q_there = seg == 0;   // (the first rows of q while the pages are looked up, later ones behind a tile)
                if (q_there && !copy_q()) break;
                for (; uniform(n < n_end); n += kCopyWarps) {
                    const int pages[2] = {entry[0], entry[1]};
                    look_up(n + kCopyWarps);
                    const Slot to = slot_of(n);
                    if (!wait_for(kEmpty + to.index, to.turn ^ 1)) break;
                    const bool look = uniform(mixed(n));
                    copy_tile(n, pages, {to.at}, {look ? bar(kRawFull + mine_of) : bar(kFull + to.index)});
                    if (!q_there && !copy_q()) break;
                    q_there = true;
                    if (!look) continue;
                    if (!wait_for(kRawFull + mine_of, looked++ & 1)) break;
                    const int live = min(kKeys, it.len - first_key(n));
                    uint32_t odd = 0;
#pragma unroll 1
                    for (int i = lane; i < S::kTile / 16; i += 32) {   // (rows of 128 bytes: the order within does not matter)
                        const uint32_t at = to.at + 16 * i;
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
                    __syncwarp();
                    if (a.box_rows == 0 || lane == 0) mbar_arrive(bar(kFull + to.index));
                    __syncwarp();
                }
                if (ok && !q_there && !copy_q()) break;
            } else if (mine_of == 0) {
                // exponent bytes of this lane's two keys, keys' and values' (256: no such key), of the tile after this one
                uint32_t next[2][2];
                auto exponents = [&](int n) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = first_key(n) + 32 * h + lane, at = key - page_of(key) * a.page_size;
                        const bool there = entry[h] >= 0 && entry[h] < a.n_pages;
                        const long long place = there ? entry[h] * a.exp_page_stride + at * a.exp_token_stride + hk * a.exp_head_stride : 0;
                        next[0][h] = there ? __ldg(a.k_exp + place) : 256u;
                        next[1][h] = there ? __ldg(a.v_exp + place) : 256u;
                    }
                };
                // of a tile: its value rows' largest exponent byte (127 without rows); bit 8: not all are near it, or a key's is one
                // with which a score times 2^exponent might leave the range of its sums
                auto reference = [&](const uint32_t (&k)[2], const uint32_t (&e)[2]) {
                    const bool far = (k[0] != 256u && k[0] - 63u > 128u) || (k[1] != 256u && k[1] - 63u > 128u);
                    const uint32_t top = __reduce_max_sync(0xffffffffu, max(e[0] == 256u ? 0u : e[0] + 1, e[1] == 256u ? 0u : e[1] + 1));
                    const uint32_t least = __reduce_min_sync(0xffffffffu, min(e[0], e[1]));
                    if (top == 0) return 127u;
                    return top - 1 - least <= static_cast<uint32_t>(kNarrow) && !__any_sync(0xffffffffu, far) ? top - 1 : top - 1 | 256u;
                };
                // (what a tile needs is asked for a tile and two tiles before)
                int n = n0, pages[2];
                look_up(n);
                pages[0] = entry[0], pages[1] = entry[1];
                exponents(n);
                look_up(n + 2);
                for (; uniform(n < n_end); n += 2) {   // keys and values of a tile lie in the same pages
                    const uint32_t exps[2][2] = {{next[0][0], next[0][1]}, {next[1][0], next[1][1]}};
                    exponents(n + 2);
                    const int following[2] = {entry[0], entry[1]};
                    look_up(n + 4);
                    const uint32_t ref = reference(exps[0], exps[1]);
                    const Slot k = slot_of(n), v = slot_of(n + 1);
                    if (!wait_for(kEmpty + k.index, k.turn ^ 1)) break;
                    if (!wait_for(kEmpty + v.index, v.turn ^ 1)) break;
                    const int tile = (n >> 1) % kInfos, raw = v.index - S::kSlotsK;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        s_kf[tile * kKeys + 32 * h + lane] = exps[0][h] == 256u ? 1.0f : pow2_of_byte(exps[0][h]);
                        s_exp[raw * kKeys + 32 * h + lane] = static_cast<uint8_t>(exps[1][h]);
                    }
                    if (lane == 0) s_info[tile] = ref;
                    __syncwarp();
                    copy_tile(n, pages, {k.at, v.at}, {bar(kFull + k.index), bar(kRawFull + raw)});
                    if (!ok) break;
                    pages[0] = following[0], pages[1] = following[1];
                }
            } else {
                if (!copy_q()) break;
                // value tiles into f16, half of the rows a warp
                constexpr int kPieces = D / 16, kStep = 32 / kPieces, kCount = kKeys / 2 * kPieces / 32;   // pieces of 16 codes
                constexpr int kBatch = std::min(kCount, 2);
                const int piece = lane % kPieces, half = 32 * (mine_of - 1), r0 = half + lane / kPieces;
                for (int n = n0 + 1; uniform(n < n_end); n += 2) {
                    const bool look = uniform(mixed(n));
                    const int live = min(kKeys, it.len - first_key(n));
                    const Slot v = slot_of(n);
                    const int raw = v.index - S::kSlotsK;
                    if (!wait_for(kRawFull + raw, v.turn)) break;
                    // f16 2^(e - that of the tile), or 1 where the softmax takes each row's own exponent
                    const uint32_t info = s_info[(n >> 1) % kInfos];
                    const int d = s_exp[raw * kKeys + half + lane] - static_cast<int>(info & 255u);
                    const float f = (info & 256u) != 0 || half + lane >= live ? 1.0f : pow2(max(d, -kNarrow));
                    const uint32_t mine = pack_f16x2(f, f);
                    const uint32_t to = v.at + (piece >> 2) * kPanel;
#pragma unroll 1
                    for (int i0 = 0; i0 < kCount; i0 += kBatch) {   // (rolled: the block's warps share one instruction cache)
                        uint4 w[kBatch];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) w[i] = lds128(raw_at<D>(v.at, (i0 + i) * kStep + r0, 16 * piece));
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            const int r = (i0 + i) * kStep + r0;
                            if (r >= live) w[i] = make_uint4(0, 0, 0, 0);
                            const uint32_t scale = __shfl_sync(0xffffffffu, mine, r & 31);
                            uint4 x, y;
                            f16_of_codes(w[i].x, scale, x.x, x.y);
                            f16_of_codes(w[i].y, scale, x.z, x.w);
                            f16_of_codes(w[i].z, scale, y.x, y.y);
                            f16_of_codes(w[i].w, scale, y.z, y.w);
                            // pieces 2 p and 2 p + 1 of the row, in the order that keeps a row's lanes in different banks
                            const bool turn = (piece & 4) != 0;
                            const int c = (2 * piece) & 7, c0 = turn ? c + 1 : c, c1 = turn ? c : c + 1;
                            sts128(to + r * 128 + ((c0 ^ (r & 7)) << 4), turn ? y : x);
                            sts128(to + r * 128 + ((c1 ^ (r & 7)) << 4), turn ? x : y);
                        }
                    }
                    if (look) {   // the warp's rows, 128 bytes of each panel
                        uint32_t odd = 0;
                        __syncwarp();
#pragma unroll 1
                        for (int i = lane; i < kKeys / 2 * (D / 8); i += 32) {
                            const uint32_t at = v.at + (i >> 8) * kPanel + half * 128 + (i & 255) * 16;
                            const uint4 x = lds128(at);
                            const uint32_t any = odd_bits_f16(x.x) | odd_bits_f16(x.y) | odd_bits_f16(x.z) | odd_bits_f16(x.w);
                            odd |= any;
                            if (any) sts128(at, make_uint4(without_odd_f16(x.x), without_odd_f16(x.y), without_odd_f16(x.z), without_odd_f16(x.w)));
                        }
                        if (odd) *s_odd = 1;
                    }
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kFull + v.index));
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
            // (f16 operands: format 0 for both)
            constexpr uint32_t kIdescS = kE4m3 ? idesc_e4m3_f32(kRowsTile, kKeys) : idesc_bf16_f32(kRowsTile, kKeys);
            constexpr uint32_t kIdescO = (idesc_bf16_f32(kRowsTile, D) | 1u << 16) & (kE4m3 ? ~(1u << 7 | 1u << 10) : ~0u);
            auto wait = [&](int i, uint32_t parity) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(i), parity, kSpinBudget));
                return ok;
            };
            for (; uniform(it.n > 0 && it.off + g0 < hi && ok); ++seg) {
                const int g1 = end_of(it), count = g1 - g0;
                for (int i = 0; uniform(i <= count && ok); ++i) {
                    const int t = tiles + i, n = 2 * t, u = t - 1, nv = n - 1;   // tile t's scores, tile u's product with the values
                    // The scores take the place of weights that the product two tiles back has read.  (Every phase of this barrier
                    // is waited for before the next but one can begin: a wait tells only neighbours apart.)
                    if (uniform(t >= 2 && (i > 0 || seg == 0))) {
                        if (!wait(kODone, t & 1)) break;
                    }
                    const Slot keys = slot_of(n), values = slot_of(max(nv, 1));
                    if (uniform(i < count) && !wait(kFull + keys.index, keys.turn)) break;
                    if (uniform(i == 0) && !wait(kQFull, seg & 1)) break;
                    tc_fence_after();
                    fence_proxy_async_shared();   // the copies were written through the generic proxy
                    if (uniform(i < count)) {
                        // (descriptors of later operands are sums: fewer instructions than from the address each time)
                        const uint32_t d = tmem + D + (t & 1) * kKeys;
                        const bool narrow_rows = kE4m3 && D == 64;
                        const uint64_t q0 = narrow_rows ? sdesc_k_sw64(smem_u32(s_q)) : sdesc_k_sw128(smem_u32(s_q));
                        const uint64_t k0 = narrow_rows ? sdesc_k_sw64(keys.at) : sdesc_k_sw128(keys.at);
                        if constexpr (kE4m3) {
#pragma unroll
                            for (int part = 0; part < 2; ++part)
#pragma unroll
                                for (int k = 0; k < D / 32; ++k)
                                    mma_e4m3_if(leader, d, q0 + (part * kRowsTile * D + (k >> 2) * (kRowsTile * 128) + (k & 3) * 32) / 16,
                                                k0 + ((k >> 2) * kPanel + (k & 3) * 32) / 16, kIdescS, part + k > 0);
                        } else {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
                                mma_if(leader, d, q0 + ((k >> 2) * (kRowsTile * 128) + (k & 3) * 32) / 16,
                                       k0 + ((k >> 2) * kPanel + (k & 3) * 32) / 16, kIdescS, k > 0);
                        }
                        commit_if(leader, bar(kEmpty + keys.index));
                        commit_if(leader, bar(kSFull + (t & 1)));
                        if (uniform(i == count - 1)) commit_if(leader, bar(kQEmpty));
                    }
                    if (uniform(i > 0)) {
                        // (the values are waited for behind the next scores: e4m3 ones are converted just in time)
                        if (!wait(kFull + values.index, values.turn)) break;
                        if (!wait(kPFull + (u & 1), (u >> 1) & 1)) break;
                        if (uniform(i == 1 && seg > 0) && !wait(kOFree, (seg - 1) & 1)) break;
                        tc_fence_after();
                        fence_proxy_async_shared();
                        const uint32_t pt = tmem + D + (u & 1) * kKeys;
                        const uint64_t v0 = sdesc_values(values.at);
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k) {
                            const uint32_t part = pt + 16 * k / S::kCut * S::kCut + 16 * k % S::kCut / 2;
                            mma_tmem_a_if(leader, tmem, part, v0 + k * 2048 / 16, kIdescO, i > 1 || k > 0);
                            mma_tmem_a_if(leader, tmem, part + S::kCut / 2, v0 + k * 2048 / 16, kIdescO, 1);
                        }
                        commit_if(leader, bar(kEmpty + values.index));
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
            for (int n = max(0, 2 * tiles - 2 * kSlots); uniform(ok && n < 2 * tiles); ++n) {   // the last uses of the slots
                const int again = n + (kE4m3 ? 2 * (n & 1 ? S::kSlotsV : S::kSlotsK) : kSlots);
                const Slot o = slot_of(n);
                if (again >= 2 * tiles) ok = __all_sync(0xffffffffu, mbar_wait(bar(kEmpty + o.index), o.turn, kSpinBudget));
            }
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
        int swaps = 0;   // buffers that have gone from half to half
        const uint32_t quarter = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        for (; it.n > 0 && it.off + g0 < hi && ok; ++seg) {
            const int g1 = end_of(it), count = g1 - g0;
            const int mtiles = it.items / a.n_kv_heads, hk = it.h / mtiles, row_at = (it.h - hk * mtiles) * kRowsTile;
            const int rows = min(kRowsTile, it.draft * group - row_at);
            const bool twice = S::kSplit && rows <= kRowsTile / 2;
            const int distinct = twice ? kRowsTile / 2 : kRowsTile, row = threadIdx.x & (distinct - 1), half = threadIdx.x / distinct;
            const bool live = row < rows, idle = (warp * 32 & (distinct - 1)) >= rows;   // idle: none of the warp's rows is a live one
            const int t_row = a.tokens_of(row_at + row), head = hk * group + (row_at + row) - t_row * group;
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
            auto sees = [&](int k0) { return seen_of(k0, from, it.ctx, seen); };
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
            float c_row = c;   // e4m3: the scale of this row's scores, apart from the keys' exponent
            // The running maximum of the scores (to 2^kSlack) with the sum of the softmax against it; O is held against
            // m_out, for e4m3 that of score + exponent of the value row, times 2^kShift.
            float m = kNone, l = 0.0f, m_out = kNone;
            for (int i = 0; i < count; ++i) {
                const int t = tiles + i, k0 = key_lo + i * kKeys;
                if (!__all_sync(0xffffffffu, mbar_wait(bar(kSFull + (t & 1)), (t >> 1) & 1, kSpinBudget))) {
                    ok = false;
                    break;
                }
                __syncwarp();   // (TMEM is read by whole, converged warps)
                tc_fence_after();
                if (!idle) {
                    const uint32_t at = quarter + D + (t & 1) * kKeys;
                    // e4m3: the keys' exponents; that of the values, as a rule one for all
                    uint32_t info = 0;
                    float cs = c, ev = 0.0f;
                    if constexpr (kE4m3) {
                        if (i == 0) c_row = fminf(fmaxf(c * pow2(s_qe[(seg & 3) * kRowsTile + row]), 1e-37f), 3e38f);   // (0 times -inf would be NaN)
                        info = s_info[t % kInfos];
                        cs = c_row;
                        ev = static_cast<float>(static_cast<int>(info & 255u) - 127);
                    }
                    const int c0 = twice ? kKeys / 2 * half : 0, c1 = twice ? c0 + kKeys / 2 : kKeys;   // the row's keys of the tile
                    const bool masked = bad || k0 < odd_from || k0 + kKeys > it.ctx;
                    uint64_t keep = ~0ULL;
                    if (masked) {
                        keep = sees(k0);
                        if (bad) keep &= resident(k0);
                    }
                    // some of the scores; -infinity where the row does not see the key
                    constexpr int kCut = S::kCut;
                    auto scores = [&](int c, uint32_t (&x)[kCut]) {
                        tmem_ld(at + c, x);
                        if constexpr (kE4m3) {
                            const float4* const kf = reinterpret_cast<const float4*>(s_kf + t % kInfos * kKeys + c);
#pragma unroll
                            for (int j = 0; j < kCut / 4; ++j) {
                                const float4 f = kf[j];
                                uint32_t* const v = &x[4 * j];
                                const Pair p0 = mul2(Pair{__uint_as_float(v[0]), __uint_as_float(v[1])}, Pair{f.x, f.y});
                                const Pair p1 = mul2(Pair{__uint_as_float(v[2]), __uint_as_float(v[3])}, Pair{f.z, f.w});
                                v[0] = __float_as_uint(p0.x), v[1] = __float_as_uint(p0.y), v[2] = __float_as_uint(p1.x), v[3] = __float_as_uint(p1.y);
                            }
                        }
                        if (masked) {
                            const uint32_t k = static_cast<uint32_t>(keep >> c);
#pragma unroll
                            for (int j = 0; j < kCut; ++j)
                                if (!(k >> j & 1u)) x[j] = 0xff800000u;
                        }
                    };
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c = c0; c < c1; c += kCut) {
                        uint32_t x[kCut];
                        scores(c, x);
                        float tops[4] = {top, -INFINITY, -INFINITY, -INFINITY};   // (four chains)
#pragma unroll
                        for (int j = 0; j < kCut; ++j) tops[j & 3] = fmaxf(tops[j & 3], __uint_as_float(x[j]));
                        top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    }
                    top *= cs;
                    float top_out = top + ev;
                    bool apart = false;   // each key with its own exponents, and the softmax's sum with an exponential of its own
                    if (kE4m3) apart = uniform((info & 256u) != 0 || fmaxf(m_out, top_out) - fmaxf(m, top) - ev > 60.0f);
                    if (kE4m3 && apart) {
                        if (twice) keep &= 0xffffffffULL << (32 * half);
                        const float2 tops = apart_maxima(a, at, keep, table, it.len, k0, hk, info, c_row);
                        top = tops.x;
                        top_out = tops.y;
                    }
                    bool raise = top > m + kSlack;
                    float f_out = 1.0f;
                    if (kE4m3) {
                        if (raise) {
                            l *= exp2_fast(m - top);
                            m = top;
                        }
                        raise = top_out > m_out + kSlack;
                        if (raise) {
                            f_out = exp2_fast(m_out - top_out);
                            m_out = top_out;
                        }
                    } else if (raise) {
                        f_out = exp2_fast(m - top);
                        l *= f_out;
                        m = m_out = top;
                    }
                    if (uniform(raise) && i > 0) {
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
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f_out);
                            tmem_st32(quarter + d, o);
                        }
                    }
                    if (kE4m3 && apart) {
                        l += apart_weights(a, at, keep, table, it.len, k0, hk, info, c_row, m, m_out);
                    } else {
                        const float off = kE4m3 ? ev + kShift - m_out : -m;
                        Pair sum = {0.0f, 0.0f};
                        const Pair by = {cs, cs}, from = {off, off};
#pragma unroll 1
                        for (int c = c0; c < c1; c += kCut) {   // in the scores' place: the first parts, two a column, then the second
                            uint32_t x[kCut], hi_part[kCut / 2], lo_part[kCut / 2];
                            scores(c, x);
#pragma unroll
                            for (int j = 0; j < kCut / 2; ++j) {
                                Pair p = fma2(Pair{__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])}, by, from);
                                p.x = exp2_fast(p.x);
                                p.y = exp2_fast(p.y);
                                sum = add2(sum, p);
                                Pair minus;
                                if constexpr (kE4m3) {
                                    hi_part[j] = pack_f16x2(p.x, p.y);
                                    const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi_part[j]));
                                    minus = {-back.x, -back.y};
                                } else {
                                    hi_part[j] = pack_bf16x2(p.x, p.y);
                                    // (signs flipped: one operation each with the shift and the mask)
                                    minus = {__uint_as_float((hi_part[j] << 16) ^ 0x80000000u), __uint_as_float((hi_part[j] & 0xffff0000u) ^ 0x80000000u)};
                                }
                                const Pair rest = add2(p, minus);
                                lo_part[j] = kE4m3 ? pack_f16x2(rest.x, rest.y) : pack_bf16x2(rest.x, rest.y);
                            }
                            tmem_st(at + c, hi_part);
                            tmem_st(at + c + kCut / 2, lo_part);
                        }
                        l += kE4m3 ? (sum.x + sum.y) * exp2_fast(-off - m) : sum.x + sum.y;
                        if (twice) {
                            const uint32_t none[16] = {0};
                            tmem_st(at + 32 * (1 - half), none);
                            tmem_st(at + 32 * (1 - half) + 16, none);
                        }
                    }
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
                // Rows that are there twice: the upper half's maxima and sum, then its O by 16 columns, to the lower half, which joins
                // them.  Four float4 [32] for each of the two pairs of warps.
                float f_mine = 1.0f, f_other = 0.0f;
                const int pair = warp & 1;
                const uint32_t swap = smem_u32(bars) + S::kBars + pair * 2048 + lane * 16;
                auto give = [&](const uint32_t (&x)[16], int n) {   // the upper half
                    ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(kSwapEmpty + pair), (swaps & 1) ^ 1, kSpinBudget));
                    if (!ok) return;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * i < n) sts128(swap + 512 * i, make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kSwapFull + pair));
                    ++swaps;
                };
                auto take = [&](uint32_t (&x)[16], int n) {   // the lower half
                    ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(kSwapFull + pair), swaps & 1, kSpinBudget));
                    if (!ok) return;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * i < n) {
                            const uint4 v = lds128(swap + 512 * i);
                            x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
                        }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kSwapEmpty + pair));
                    ++swaps;
                };
                if (twice) {
                    uint32_t u[16] = {__float_as_uint(m), __float_as_uint(l), __float_as_uint(m_out)};
                    if (half == 1) {
                        give(u, 4);
                    } else {
                        take(u, 4);
                        const float m1 = __uint_as_float(u[0]), l1 = __uint_as_float(u[1]), out1 = __uint_as_float(u[2]);
                        const float both = fmaxf(m, m1), both_out = fmaxf(m_out, out1);
                        l = l * exp2_fast(m - both) + l1 * exp2_fast(m1 - both);
                        f_mine = exp2_fast(m_out - both_out);
                        f_other = exp2_fast(out1 - both_out);
                        m = both;
                        m_out = both_out;
                    }
                }
                // (what O is held against, as a power of two over the sum's)
                const float over = kE4m3 ? m_out - kShift - m : 0.0f;
                const float inv = l > 0.0f ? (kE4m3 ? exp2_fast(within(over)) : 1.0f) / l : (l == 0.0f ? 0.0f : NAN);
                float odd_out = 0.0f;   // bf16: NaN once an output's product was NaN or an infinity
                __nv_bfloat16* const out = a.out + static_cast<long long>(it.row0 + t_row) * a.out_token_stride + static_cast<long long>(head) * a.out_head_stride;
#pragma unroll 1
                for (int d = 0; d < D; d += 16) {
                    uint32_t o[16];
                    tmem_ld(quarter + d, o);
                    if (twice) {
                        if (half == 1) {
                            give(o, 16);
                        } else {
                            uint32_t other[16] = {};
                            take(other, 16);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                o[j] = __float_as_uint(fmaf(__uint_as_float(o[j]), f_mine, __uint_as_float(other[j]) * f_other));
                        }
                        if (half == 1) continue;
                    }
                    if (!kE4m3) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) odd_out = fmaf(__uint_as_float(o[j]), 0.0f, odd_out);
                    }
                    if (kE4m3 && whole && uniform(over < kLeast)) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * rest_of(over));
                    }
                    if (live && whole) {   // (the upper half of rows that are there twice is through)
#pragma unroll
                        for (int u = 0; u < 16; u += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                w[j] = pack_bf16x2(__uint_as_float(o[u + 2 * j]) * inv, __uint_as_float(o[u + 2 * j + 1]) * inv);
                            *reinterpret_cast<uint4*>(out + d + u) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else if (live) {   // [4 columns][row]: whole lines
#pragma unroll
                        for (int u = 0; u < 16; u += 4)
                            reinterpret_cast<uint4*>(part)[((d + u) >> 2) * kRowsTile + row] = make_uint4(o[u], o[u + 1], o[u + 2], o[u + 3]);
                    }
                    __syncwarp();   // TMEM is read by whole warps
                }
                if (*s_odd != 0 && live && half == 0 && !(whole && l == 0.0f))
                    add_odd<D, kE4m3>(a, table, whole ? out : nullptr, part + row * 4, key_lo, key_hi, odd_from, it.ctx, from, hk, seen);
                if constexpr (!kE4m3) {
                    const bool mine = odd_out != 0.0f && live && half == 0;
                    if (uniform(mine && l == l))
                        settle_odd<D>(a, table, whole ? out : nullptr, part + row * 4, key_lo, key_hi, it.ctx, from, hk, seen, mine && l == l, whole && l == 0.0f);
                }
                if (live && half == 0 && whole && a.lse)
                    a.lse[static_cast<long long>(it.row0 + t_row) * a.n_heads + head] = l == 0.0f ? -INFINITY : fmaf(m, kLn2, logf(l));
                if (live && half == 0 && !whole) reinterpret_cast<float4*>(part + kRowsTile * D)[row] = make_float4(m, l, kE4m3 ? m_out - kShift : m, 0.0f);
                if (threadIdx.x == 0 && whole && a.by_item > 0 && !uncut) headers[it.ordinal].last = -1;
                if (threadIdx.x == 0 && g0 == 0 && !whole) {
                    Header h;
                    h.first = blockIdx.x;
                    h.b = it.b;
                    h.hk = hk;
                    h.first_row = row_at;
                    h.rows = rows;
                    h.last = static_cast<int>(quotient(it.off + it.n - 1, run));
                    headers[a.by_item > 0 ? it.ordinal : static_cast<int>(blockIdx.x)] = h;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kOFree));
            tiles += count;
            next_item(a, it);
            g0 = 0;
        }
        if (!ok) {
            record_error(a.status, MOE_ERR_TIMEOUT);
            if (threadIdx.x == 0 && a.by_item > 0 && !uncut) give_up(a, headers, it, g0, hi);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kProductWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kCols);
    }
}

// ---------------------------------------------------------------- the join

// Block (x, y): header x's item; 32 of its rows, and 32 columns of them.
template <int D>
__global__ void __launch_bounds__(256) tree_attention_join_kernel(const TreeArgs a)
{
    using S = Shape<D, false>;
    wait_for_previous();
    const Header h = reinterpret_cast<const Header*>(static_cast<const char*>(a.ws) + kTreeCtrlBytes)[blockIdx.x];
    const int row0 = (blockIdx.y & 3) * 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (h.last < 0 || row0 >= h.rows) return;
    const int row = row0 + lane, col4 = (blockIdx.y >> 2) * 8 + warp;   // four columns
    const int parts = h.last - h.first + 1;
    const float* const base = reinterpret_cast<const float*>(static_cast<const char*>(a.ws) + kTreeCtrlBytes + sizeof(Header) * kMaxBlocks);
    auto part = [&](int i) { return base + (2LL * (h.first + i) + (i == 0 ? 1 : 0)) * S::kPart; };
    float m = kNone, m_out = -INFINITY;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float4 q = reinterpret_cast<const float4*>(part(i) + kRowsTile * D)[row];
        m = fmaxf(m, q.x);
        m_out = fmaxf(m_out, q.z);
    }
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float4 q = reinterpret_cast<const float4*>(part(i) + kRowsTile * D)[row];
        const float4 x = reinterpret_cast<const float4*>(part(i))[col4 * kRowsTile + row];
        // (never 0: an infinity that the row sees is one whatever its part's weight.  What that adds of a finite O is less than
        // the exponential's own flush takes away.)
        const float f = fmaxf(exp2_fast(q.z - m_out), 0x1p-149f);
        l = fmaf(q.y, exp2_fast(q.x - m), l);
        o.x = fmaf(x.x, f, o.x);
        o.y = fmaf(x.y, f, o.y);
        o.z = fmaf(x.z, f, o.z);
        o.w = fmaf(x.w, f, o.w);
    }
    if (row >= h.rows) return;
    const float inv = l > 0.0f ? exp2_fast(within(m_out - m)) / l : (l == 0.0f ? 0.0f : NAN), rest = rest_of(m_out - m);
    if (l == 0.0f) o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);   // no score above -infinity, whatever the values
    const int group = a.n_heads / a.n_kv_heads, t = (h.first_row + row) / group, head = h.hk * group + (h.first_row + row) - t * group;
    const long long token = a.row_start[h.b] + t;
    *reinterpret_cast<uint2*>(a.out + token * a.out_token_stride + head * a.out_head_stride + 4 * col4) =
        make_uint2(pack_bf16x2(o.x * rest * inv, o.y * rest * inv), pack_bf16x2(o.z * rest * inv, o.w * rest * inv));
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
    auto encode = [&](CUtensorMap* map, const void* rows_of, CacheBox box) {
        return encode_cache_map(map, rows_of, box, D, a.page_size, a.n_kv_heads, a.n_pages, a.token_bytes, a.head_bytes, a.page_bytes, rows);
    };
    a.box_rows = rows >= 8 && encode(&map_k, a.k, kE4m3 ? kCodesSwizzled : kBf16Swizzled) && encode(&map_v, a.v, kE4m3 ? kCodes : kBf16Swizzled)
                     ? rows : 0;
    const unsigned grid = static_cast<unsigned>(S::kCtas * std::min(num_sms(), kMaxSms));
    // at most so many items while no row is in two sequences: every sequence has one row tile a key head, and one more per 128 rows
    const long long items = static_cast<long long>(a.n_kv_heads) * (a.B + static_cast<long long>(a.T) * (a.n_heads / a.n_kv_heads) / kRowsTile);
    a.by_item = items <= grid ? static_cast<int>(items) : 0;
    kernel<<<grid, kThreads, S::kSmem, s>>>(map_k, map_v, a);
    const cudaError_t launched = cudaGetLastError();
    if (launched != cudaSuccess) return launched;
    return launch_after(tree_attention_join_kernel<D>, dim3(a.by_item > 0 ? static_cast<unsigned>(a.by_item) : grid, 4 * D / 32), 256, 0, s, a);
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
    // row / group for the at most 2^16 rows of a key head: with mul = 2^32 / group rounded up, row * (mul * group - 2^32) < 2^32
    const uint32_t group = static_cast<uint32_t>(a.n_heads / a.n_kv_heads);
    a.group_mul = group > 1 ? static_cast<uint32_t>(((1ULL << 32) + group - 1) / group) : 0;
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
