// logprobs.cu -- log probabilities of given tokens, entropy and the most likely
// alternatives, read off a row of logits, and their gradient.
//
// Forward.  A row is read once from memory, by one block or, when there are few
// rows, by a cluster of up to 8 whose parts meet in distributed shared memory.
// A thread keeps the running maximum m of what it has read and, against it,
//   l = sum 2^z,  w = sum 2^z z,  z = (x - m) log2 e,
// so that lse = m + ln l and entropy = ln l - ln 2 * w / l: sums of terms of one
// sign, whatever the size of the logits (z as it is computed has a known rounding of
// m log2 e in it, which is taken out again: Stats).
// Alternatives: no list is kept while streaming, only the maximum of every few
// pieces that a thread reads.  From the threads' maxima comes a threshold that at
// least n values reach; the pieces whose maximum reaches it -- some dozens, still
// in L2 -- are read again, and the values found are ranked by counting how many
// exceed each (keys of value and index are distinct, so the ranks are too).
// Backward: element by element, from lse and entropy.
//
// Measured (6801 GB/s copied): 4096 x 131072 fp32 with the 5 best, 2147 MB read in
// 312 us (1.01 of the copy rate); 2047 x 50257 bf16 with the 20 best, 206 MB in 43 us
// (0.70); the gradient of 4096 x 50257 bf16, 823 MB in 119 us (1.02).  fp32 rows and
// gradients are bound by memory; bf16 rows by instructions as well (some 50 for the 8
// values of a piece: unpack, raise, fma, ex2, add, fma) and by what a row waits for.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;      // of a block that reads a row or its share; fewer for a short row of many, more for a
constexpr int kFewThreads = 64, kMoreThreads = 512;   // long one of some hundreds
constexpr int kMostWarps = kMoreThreads / 32;
constexpr int blocks_of(int threads) { return threads == kThreads ? 5 : (threads == kMoreThreads ? 2 : 16); }   // per SM
constexpr int kBatch = 4;          // 16-byte pieces that a thread has in flight
constexpr int kMaxima = 2048;       // maxima kept of a row, at most 2048 / readers per reader
constexpr int kMaxFound = 1024;    // values at or above the threshold that are ranked at once
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Values are raised to this: their exponentials are 0 all the same, and 0 times them is 0 (-inf would make NaN).
constexpr float kFloor = -1e30f;
constexpr float kNear = 0x1p24f;   // the largest |maximum| against which a row's values are taken in one fma

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two floats of a packed instruction, each rounded as a single one's.
struct Pair {
    float x, y;
};
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ Pair add(Pair a, Pair b)
{
    Pair r;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// max that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Ascending in the value; -0 counts as +0, NaN below everything (0).
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    if (x != x) return 0u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t order)
{
    if (order == 0u) return NAN;
    return __uint_as_float(order & 0x80000000u ? order ^ 0x80000000u : ~order);
}
// Distinct keys: larger value first, then lower index.
__device__ __forceinline__ uint64_t key_of(uint32_t order, int i)
{
    return (static_cast<uint64_t>(order) << 32) | static_cast<uint32_t>(~i);
}

template <class T>
struct Piece;
template <>
struct Piece<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ uint4 nothing() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    static __device__ __forceinline__ void unpack(const uint4 v, float (&x)[4])
    {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
    // each value raised to kFloor, NaN kept
    static __device__ __forceinline__ uint4 floored(const uint4 v)
    {
        auto f = [](uint32_t w) { return __float_as_uint(max_nan(__uint_as_float(w), kFloor)); };
        return make_uint4(f(v.x), f(v.y), f(v.z), f(v.w));
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    static __device__ __forceinline__ float at(const uint4 v, int i)
    {
        return __uint_as_float(i & 2 ? (i & 1 ? v.w : v.z) : (i & 1 ? v.y : v.x));
    }
    static __device__ __forceinline__ float top(const uint4 v)
    {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
};
template <>
struct Piece<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ uint4 nothing() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    static __device__ __forceinline__ void unpack(const uint4 v, float (&x)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 floored(const uint4 v)
    {
        const __nv_bfloat162 low = __float2bfloat162_rn(kFloor);
        auto f = [&](uint32_t w) {
            const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w), low);
            return *reinterpret_cast<const uint32_t*>(&r);
        };
        return make_uint4(f(v.x), f(v.y), f(v.z), f(v.w));
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8])
    {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    static __device__ __forceinline__ float at(const uint4 v, int i)
    {
        const uint32_t w = i & 4 ? (i & 2 ? v.w : v.z) : (i & 2 ? v.y : v.x);
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
    static __device__ __forceinline__ float top(const uint4 v)
    {
        const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
        const __nv_bfloat162 t = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
        return fmaxf(__bfloat162float(t.x), __bfloat162float(t.y));
    }
};

// A row as whole 16-byte pieces and the few values before and behind them.
template <class T>
struct Row {
    const T* x;          // value 0
    const uint4* body;   // piece 0
    int head, pieces;    // values before piece 0; pieces
    __device__ __forceinline__ Row(const void* logits, long long row_stride, long long row, int vocab)
    {
        constexpr int kN = Piece<T>::kN;
        x = static_cast<const T*>(logits) + row * row_stride;
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(T) % kN);
        head = min(off ? kN - off : 0, vocab);
        body = reinterpret_cast<const uint4*>(x + head);
        pieces = (vocab - head) / kN;
    }
    // the edge value of thread t (fewer than 2 kN of them), or -1
    __device__ __forceinline__ int edge(int t, int vocab) const
    {
        const int i = t < head ? t : head + pieces * Piece<T>::kN + (t - head);
        return i < vocab ? i : -1;
    }
};

// The running statistics of one thread, warp, block or cluster.
struct Stats {
    float m, l, w;   // maximum, sum 2^z, sum 2^z z with z = (x - m) log2 e + off(m)
    // z = x log2 e - base(m) in one fma, while |m| <= kNear.  The base's rounding off(m) is in every z, up to |m| log2 e
    // 2^-24: 7e-4 at 10^4.  Maxima are raised and log probabilities taken with it, so that it costs neither anything.
    // Past kNear it would be more than an exponential can hold (from some 1e9 on: finite masks until something else is
    // read, rows of nothing else), and the base overflows at the type's lowest value: there the difference comes first.
    static __device__ __forceinline__ bool is_far(float v) { return fabsf(v) > kNear && fabsf(v) < INFINITY; }
    static __device__ __forceinline__ float base_of(float v) { return __fmul_rn(v, kLog2e); }
    static __device__ __forceinline__ float off(float v) { return fabsf(v) <= kNear ? fmaf(v, kLog2e, -base_of(v)) : 0.0f; }
    __device__ __forceinline__ bool far() const { return is_far(m); }
    __device__ __forceinline__ float base() const { return base_of(m == -INFINITY ? 0.0f : m); }
    __device__ __forceinline__ void raise_by(float d, float to)
    {
        d = fmaxf(d, -1e20f);
        const float f = exp2_fast(d);
        w = f * (w + d * l);
        l *= f;
        m = to;
    }
    // to >= m, neither far
    __device__ __forceinline__ void raise_near(float to)
    {
        if (to > m) raise_by(base_of(m) - base_of(to), to);
    }
    __device__ __forceinline__ void raise(float to)   // to >= m
    {
        if (to > m) raise_by(fmaf(m - to, kLog2e, off(to) - off(m)), to);
    }
    // The warp's, in every lane: the maximum first, then plain sums.
    __device__ __forceinline__ void join_warp()
    {
        float to = m;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, off));
        if (__any_sync(0xffffffffu, is_far(m) || is_far(to)))
            raise(to);
        else
            raise_near(to);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            l += __shfl_xor_sync(0xffffffffu, l, off);
            w += __shfl_xor_sync(0xffffffffu, w, off);
        }
    }
    // one value, against any maximum
    __device__ __forceinline__ void add(float x)
    {
        const float z = max_nan(far() ? (x - m) * kLog2e : fmaf(x, kLog2e, -base()), kFloor), e = exp2_fast(z);
        l += e;
        w = fmaf(e, z, w);
    }
};

// What the search for the best keys of a row needs beside the maxima and room for kMaxFound keys.  Shared memory is
// kept small, since what it leaves of the SM's 256 KB holds the loads in flight (with 33 KB a block 4096 x 131072
// fp32 rows took 377 us instead of 325).
struct Finder {
    uint64_t best[MOE_MAX_TOP];     // the block's best keys, in order
    uint32_t least[kMostWarps];
    int entries, found, before[kMostWarps];
    uint16_t entry[kMaxima];
};

template <class T>
struct Shared {
    Stats stats[kMostWarps];
    Finder f;
    union {
        T top[kMaxima];                            // until the entries are listed
        alignas(16) uint64_t keys[kMaxFound];      // from then on
    };
};

constexpr int kStreamBlocks = 4; // blocks per SM of the streaming kernel,
constexpr int kReaders = 256;    // their threads that read rows
constexpr int kFinishers = 64;  // and that finish them
template <class T>
struct StreamShared {
    Stats stats[2][kReaders / 32];
    Finder f;
    T top[2][kMaxima];
    alignas(16) uint64_t keys[kMaxFound];
};

// Named barriers of the streaming kernel: of the finishers; rows handed over and taken (one each per buffer).
enum Barrier : int { kBarFinish = 1, kBarFull = 2, kBarEmpty = 4 };
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// A barrier of the NT threads that look for the best: the block, or its finishers.
template <int NT>
__device__ __forceinline__ void sync_finders()
{
    bar_sync(kBarFinish, NT);
}

// How many of the pairs part, part + kParts, .. of keys[0, count) (16-byte aligned) exceed key.
template <int kParts>
__device__ __forceinline__ int rank_in(const uint64_t* keys, int count, uint64_t key, int part)
{
    int rank = 0;
#pragma unroll 8
    for (int i = 2 * part; i < count; i += 2 * kParts) {
        const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(keys + i);
        rank += (k.x > key) + (i + 1 < count && k.y > key);
    }
    return rank;
}

// Maxima are kept in the logits' type.  Where a finder looks at several readers' bf16 maxima, two share a word: those of
// readers r and r + R / 2.
template <class T, int NT, int R>
constexpr int maxima_in_a_word = sizeof(T) == 2 && R >= 2 * NT ? 2 : 1;
template <class T, int NT, int R>
__device__ __forceinline__ int maximum_place(int reader)
{
    return maxima_in_a_word<T, NT, R> == 2 ? reader % (R / 2) * 2 + reader / (R / 2) : reader;
}

// The best n keys of pieces [lo, hi) of a row and the edge values into s.best (0 where there are none), sorted: by
// NT threads, from the maxima of the groups of pieces that R readers took.
template <class T, int NT, int R, bool kBeam>
__device__ void find_best(Finder& s, const T* tops, uint64_t* keys, const Row<T>& row, int n, int lo, int hi,
                          int per_group, int groups, int t, int edge, float edge_value)
{
    constexpr int kN = Piece<T>::kN, kNTWarps = NT / 32;
    const int lane = t & 31, warp = t >> 5;
    float thread_top = -INFINITY;
    // a thread looks at kWords words a group, of kWide maxima each
    constexpr int kWide = maxima_in_a_word<T, NT, R>, kWords = R / NT / kWide, kPer = kWords * kWide;
    static_assert(R % (NT * kWide) == 0, "equal shares");
    auto reader = [&](int c) { return c / kWide * NT + t + c % kWide * (R / 2); };
    auto maxima = [&](int g, float (&x)[kPer]) {
#pragma unroll
        for (int c = 0; c < kWords; ++c) {
            if constexpr (kWide == 2) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(tops + g * R + 2 * (c * NT + t));
                x[2 * c] = __uint_as_float(w << 16);
                x[2 * c + 1] = __uint_as_float(w & 0xffff0000u);
            } else {
                x[c] = static_cast<float>(tops[g * R + c * NT + t]);
            }
        }
    };
    for (int g = 0; g < groups; ++g) {
        float x[kPer];
        maxima(g, x);
#pragma unroll
        for (int c = 0; c < kPer; ++c) thread_top = fmaxf(thread_top, x[c]);
    }
    if (t < MOE_MAX_TOP) s.best[t] = 0;
    if (t == 0) s.entries = s.found = 0;
    // threshold: with k = ceil(n / full warps), the least of the full warps' k-th largest thread maxima is
    // reached by at least n values (a warp is full when each of its threads has maxima of something read)
    const int full = min((hi - lo) / 32, kNTWarps);
    uint32_t mine = order_of(thread_top), kth = 0xffffffffu;
    if (warp < full) {
        for (int k = (n + full - 1) / full; k > 0; --k) {
            kth = __reduce_max_sync(0xffffffffu, mine);
            const uint32_t who = __ballot_sync(0xffffffffu, mine == kth);
            if (lane == __ffs(who) - 1) mine = 0;
        }
    }
    if (lane == 0) s.least[warp] = kth;
    sync_finders<NT>();
    uint32_t level = full ? 0xffffffffu : 0u;
    for (int w = 0; w < full; ++w) level = min(level, s.least[w]);
    // compared as values: NaN never reaches the level, unless that is 0 and takes everything
    const float level_value = value_of(level);
    const bool any = level == 0u;
    // Beams: fewer than n threads with anything but masked values, which are no candidates; those above are looked for at
    // once (64 x 8 rows of 131072 fp32, one in twenty masked but for a value: 50 us, 132 when the masked ones were counted).
    const bool masked = kBeam && level_value == -INFINITY;
    // the maxima that reach it, listed warp by warp
    static_assert(kMaxima / NT <= 32, "a bit per maximum of a thread");
    uint32_t hits = 0;
    for (int g = 0; g < groups; ++g) {
        float x[kPer];
        maxima(g, x);
        uint32_t some = 0;
#pragma unroll
        for (int c = 0; c < kPer; ++c) some |= (any || (masked ? x[c] > level_value : x[c] >= level_value)) ? 1u << c : 0u;
        hits |= some << (g * kPer);
    }
    const int hit_count = __popc(hits);
    int at = hit_count;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, at, off);
        if (lane >= off) at += o;
    }
    int begin = 0;
    if (lane == 31) begin = atomicAdd(&s.entries, at);
    at += __shfl_sync(0xffffffffu, begin, 31) - hit_count;
    for (; hits; hits &= hits - 1) {
        const int k = __ffs(hits) - 1;
        s.entry[at++] = static_cast<uint16_t>(k / kPer * R + reader(k % kPer));
    }
    sync_finders<NT>();
    const int entries = s.entries;
    // (one more pass, for the values above the level alone, when those at it are too many to rank)
    int strict = masked ? 1 : 0;
    for (;; ++strict) {
        auto reaches = [&](float x) { return any || (strict ? x > level_value : x >= level_value); };
        // the entries' pieces, one per thread and step (a batch's to neighbours), four steps' loads in flight
        constexpr int kStep = NT / kBatch;
        for (int b = 0; b < per_group; ++b) {
            for (int e0 = t / kBatch; e0 < entries; e0 += 4 * kStep) {
                uint4 v[4];
                int first[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = e0 + j * kStep, e = at < entries ? s.entry[at] : 0;
                    const int piece = lo + e % R + R * ((e / R * per_group + b) * kBatch + t % kBatch);
                    first[j] = at < entries && piece < hi ? row.head + piece * kN : -1;
                    v[j] = first[j] >= 0 ? __ldg(row.body + piece) : Piece<T>::nothing();
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (first[j] < 0 || !reaches(Piece<T>::top(v[j]))) continue;
                    float x[kN];
                    Piece<T>::unpack(v[j], x);
                    uint32_t which = 0;
#pragma unroll
                    for (int i = 0; i < kN; ++i) which |= reaches(x[i]) ? 1u << i : 0u;
                    int place = atomicAdd(&s.found, __popc(which));
                    for (; which; which &= which - 1, ++place) {   // one, as a rule
                        const int i = __ffs(which) - 1;
                        if (place < kMaxFound) keys[place] = key_of(order_of(Piece<T>::at(v[j], i)), first[j] + i);
                    }
                }
            }
        }
        if (edge >= 0 && reaches(edge_value)) {
            const int place = atomicAdd(&s.found, 1);
            if (place < kMaxFound) keys[place] = key_of(order_of(edge_value), edge);
        }
        sync_finders<NT>();
        if (s.found <= kMaxFound || strict) break;
        sync_finders<NT>();
        if (t == 0) s.found = 0;
        sync_finders<NT>();
    }
    const int found = s.found;
    if (found <= kMaxFound) {
        // four lanes to a key, each with a quarter of the comparisons
        for (int a0 = 0; a0 < found; a0 += NT / 4) {
            const int a = a0 + t / 4;
            const uint64_t key = a < found ? keys[a] : ~0ull;
            int rank = rank_in<4>(keys, found, key, t & 3);
            rank += __shfl_xor_sync(0xffffffffu, rank, 1);
            rank += __shfl_xor_sync(0xffffffffu, rank, 2);
            if (a < found && (t & 3) == 0 && rank < n) s.best[rank] = key;
        }
        sync_finders<NT>();
        // fewer than n: the values at the level when those above it alone were ranked, then (level = that of
        // -inf) the NaNs, each in the order of their indices
        int have = masked ? n : found;
        for (int pass = strict ? 0 : 1; pass < 2 && have < n; ++pass) {
            const uint32_t want = pass == 0 ? level : 0u;
            if (pass == 1 && level == 0u) break;   // they were ranked with the rest
            const int steps = (hi - lo + NT - 1) / NT;
            // the edge values before the body, the body, the edge values behind it
            for (int step = -1; step <= steps && have < n; ++step) {
                const int piece = lo + step * NT + t;
                const bool side = step < 0 || step == steps;
                int count = 0;
                if (side)
                    count = edge >= 0 && (edge < row.head) == (step < 0) && order_of(edge_value) == want;
                else if (piece < hi)
                    for (int j = 0; j < kN; ++j) count += order_of(static_cast<float>(row.x[row.head + piece * kN + j])) == want;
                int incl = count;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += o;
                }
                if (lane == 31) s.before[warp] = incl;
                sync_finders<NT>();
                int at = have + incl - count;
                for (int w = 0; w < kNTWarps; ++w) {
                    if (w < warp) at += s.before[w];
                    have += s.before[w];
                }
                if (side && count && at < n) s.best[at] = key_of(want, edge);
                if (!side && count)
                    for (int j = 0; j < kN && at < n; ++j) {
                        const int i = row.head + piece * kN + j;
                        if (order_of(static_cast<float>(row.x[i])) == want) s.best[at++] = key_of(want, i);
                    }
                sync_finders<NT>();
            }
        }
        return;
    }
    // too many values above a loose threshold (a row laid out against it): n rounds over the share
    uint64_t last = ~0ull;
    for (int k = 0; k < n; ++k) {
        uint64_t best = 0;
        auto see = [&](float x, int i) {
            const uint64_t key = key_of(order_of(x), i);
            if (key < last && key > best) best = key;
        };
        for (int p = lo + t; p < hi; p += NT)
            for (int j = 0; j < kN; ++j) see(static_cast<float>(row.x[row.head + p * kN + j]), row.head + p * kN + j);
        if (edge >= 0) see(edge_value, edge);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            const uint64_t o = __shfl_xor_sync(0xffffffffu, best, off);
            best = o > best ? o : best;
        }
        if (lane == 0) keys[warp] = best;
        sync_finders<NT>();
        for (int w = 0; w < kNTWarps; ++w) best = keys[w] > best ? keys[w] : best;
        sync_finders<NT>();
        if (t == 0) s.best[k] = best;
        last = best;
    }
    sync_finders<NT>();
}

// One thread's part of pieces [lo, hi) of a row: its statistics, and with kTop the maxima of its groups of pieces, every
// R places from `tops` on.
template <class T, bool kTop, int R>
__device__ __forceinline__ Stats read_pieces(const Row<T>& row, int lo, int hi, int t, int batches, int per_group, T* tops)
{
    constexpr int kN = Piece<T>::kN;
    Stats st{-INFINITY, 0.0f, 0.0f};
    float group_top = -INFINITY;
    bool far = false;   // st.far()
    auto work = [&](const auto& v) {
        constexpr int kPieces = sizeof(v) / 16;
        float top = Piece<T>::top(v[0]);
#pragma unroll
        for (int j = 1; j < kPieces; ++j) top = fmaxf(top, Piece<T>::top(v[j]));
        if (kTop) group_top = fmaxf(group_top, top);
        const float to = fmaxf(st.m, top);
        const bool was_far = far;
        far = Stats::is_far(to);
        if (!(far || was_far)) {
            st.raise_near(to);
            const float minus_base = -st.base();
            // two sums each, of even and odd places, in packed pairs: one instruction for two values
            Pair l = {st.l, 0.0f}, w = {st.w, 0.0f};
            const Pair log2e = {kLog2e, kLog2e}, from = {minus_base, minus_base};
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                float x[kN];
                Piece<T>::unpack(Piece<T>::floored(v[j]), x);
#pragma unroll
                for (int i = 0; i < kN; i += 2) {
                    const Pair z = fma(Pair{x[i], x[i + 1]}, log2e, from), e = {exp2_fast(z.x), exp2_fast(z.y)};
                    l = add(l, e);
                    w = fma(e, z, w);
                }
            }
            st.l = l.x + l.y;
            st.w = w.x + w.y;
        } else {
            st.raise(to);
            Pair l = {st.l, 0.0f}, w = {st.w, 0.0f};
            const float minus_m = far ? -st.m : 0.0f, minus_base = far ? 0.0f : -st.base();
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                float x[kN];
                Piece<T>::unpack(v[j], x);
#pragma unroll
                for (int i = 0; i < kN; i += 2) {
                    const Pair d = fma(add(Pair{x[i], x[i + 1]}, Pair{minus_m, minus_m}), Pair{kLog2e, kLog2e}, Pair{minus_base, minus_base});
                    const Pair z = {max_nan(d.x, kFloor), max_nan(d.y, kFloor)}, e = {exp2_fast(z.x), exp2_fast(z.y)};
                    l = add(l, e);
                    w = fma(e, z, w);
                }
            }
            st.l = l.x + l.y;
            st.w = w.x + w.y;
        }
    };
    auto close_group = [&]() {
        *tops = static_cast<T>(group_top);
        tops += R;
        group_top = -INFINITY;
    };
    const uint4* src = row.body + lo + t;
    const int full = (hi - lo) / (R * kBatch);   // batches without a missing piece
    for (int b = 0, in_group = 0; b < full; ++b) {
        uint4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) v[j] = __ldg(src + j * R);
        src += R * kBatch;
        work(v);
        if (kTop && (++in_group == per_group || b + 1 == batches)) {
            close_group();
            in_group = 0;
        }
    }
    if (full < batches) {   // piece by piece: the last batch may hold few
        const int rest = hi - lo - full * R * kBatch;
        for (int j = 0; j < rest; j += R) {
            uint4 v[1] = {j + t < rest ? __ldg(src + j) : Piece<T>::nothing()};
            work(v);
        }
        if (kTop) close_group();
    }
    return st;
}

// Batches under one maximum of a reader.
template <int R>
__device__ __forceinline__ int per_maximum(int batches)
{
    return (batches + kMaxima / R - 1) / (kMaxima / R);
}

// The given token of row r, or -1 (also for one that is out of range, which is recorded).
__device__ __forceinline__ int given_token(const LogprobArgs& a, long long r)
{
    const int token = a.token[r];
    if (token >= a.vocab) record_error(a.status, MOE_ERR_INDEX);
    return token >= a.vocab ? -1 : token;
}

// What the outputs of a row take from its statistics; kBeam: the values themselves, with the maximum and sum beside them.
template <bool kBeam>
struct Result {
    bool none;            // nothing but -inf in the row
    float ref, log_l;     // log_l: ln sum e^(x - ref)
    __device__ __forceinline__ explicit Result(const Stats& s)
        : none(s.m == -INFINITY && s.l == 0.0f), ref(s.m == -INFINITY ? 0.0f : s.m), log_l(fmaf(-Stats::off(s.m), kLn2, logf(s.l)))
    {
    }
    // 2^-off, to a rounding or two
    static __device__ __forceinline__ float unturned(float off)
    {
        const float y = off * kLn2;
        return fabsf(y) < 1e-3f ? fmaf(y, fmaf(y, 0.5f, -1.0f), 1.0f) : exp2f(-off);
    }
    __device__ __forceinline__ float logprob(float x) const { return none ? -INFINITY : x - ref - log_l; }
    // by one thread
    __device__ __forceinline__ void write(const LogprobArgs& a, long long r, const Stats& s, int token, float given) const
    {
        if (s.l != s.l) record_error(a.status, MOE_ERR_NONFINITE);
        if (kBeam) a.stats[r] = make_float2(ref, s.l * unturned(Stats::off(s.m)));
        if (a.lse) a.lse[r] = ref + log_l;
        if (a.entropy) a.entropy[r] = none ? 0.0f : logf(s.l) - s.w / s.l * kLn2;   // (the same off(m) in both)
        if (a.logprob) a.logprob[r] = token < 0 ? 0.0f : logprob(given);
    }
    __device__ __forceinline__ void write_top(const LogprobArgs& a, long long r, int at, uint64_t key) const
    {
        a.top_ids[r * a.n_top + at] = key ? static_cast<int>(~static_cast<uint32_t>(key)) : -1;
        const float x = value_of(static_cast<uint32_t>(key >> 32));
        a.top_logprobs[r * a.n_top + at] = key ? (kBeam ? x : logprob(x)) : -INFINITY;
    }
};

// A row to a block of NT threads, or to a cluster of a.split blocks.
template <class T, bool kTop, int NT, bool kBeam>
__global__ void __launch_bounds__(NT, blocks_of(NT)) token_logprobs_kernel(const LogprobArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    Shared<T>& s = *reinterpret_cast<Shared<T>*>(smem);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int rank = static_cast<int>(blockIdx.x) & (a.split - 1);
    const long long r = blockIdx.x / static_cast<unsigned>(a.split);
    const Row<T> row(a.logits, a.row_stride, r, a.vocab);
    // this block's share of the pieces
    const int share = (row.pieces + a.split - 1) / a.split;
    const int lo = min(row.pieces, rank * share), hi = min(row.pieces, lo + share);
    const int batches = (hi - lo + NT * kBatch - 1) / (NT * kBatch);
    const int per_group = per_maximum<NT>(batches);
    // asked for early: the given token and its logit
    int token = -1;
    float given = 0.0f;
    if (a.logprob && rank == 0 && t == 0) {
        token = given_token(a, r);
        if (token >= 0) given = static_cast<float>(row.x[token]);
    }
    Stats st = read_pieces<T, kTop, NT>(row, lo, hi, t, batches, per_group, s.top + maximum_place<T, NT, NT>(t));
    // the values beside the whole pieces: rank 0's threads, one each
    const int edge = rank == 0 ? row.edge(t, a.vocab) : -1;
    const float edge_value = edge >= 0 ? static_cast<float>(row.x[edge]) : -INFINITY;
    if (edge >= 0) {
        st.raise(fmaxf(st.m, edge_value));
        st.add(edge_value);
    }
    st.join_warp();
    if (lane == 0) s.stats[warp] = st;
    if (kTop) {
        const int groups = per_group ? (batches + per_group - 1) / per_group : 0;
        find_best<T, NT, NT, kBeam>(s.f, s.top, s.keys, row, a.n_top, lo, hi, per_group, groups, t, edge, edge_value);
    }
    if (a.split > 1)
        cluster_sync_all();
    else
        __syncthreads();
    if (rank == 0 && (warp == 0 || a.split > 1)) {   // (without a split the first warp does the rest)
        // the row's statistics, by every warp for itself: lane i has warp i % kOwn of block i / kOwn, then the next ones
        Stats all{-INFINITY, 0.0f, 0.0f};
        constexpr int kOwn = NT / 32;
        for (int i = lane; i < a.split * kOwn; i += 32) {
            const uint32_t at = map_to_rank(smem_u32(&s.stats[i % kOwn]), i / kOwn);
            Stats o{ld_cluster_f32(at), ld_cluster_f32(at + 4), ld_cluster_f32(at + 8)};
            const float to = fmaxf(all.m, o.m);
            all.raise(to);
            o.raise(to);
            all.l += o.l;
            all.w += o.w;
        }
        all.join_warp();
        const Result<kBeam> res(all);
        if (t == 0) res.write(a, r, all, token, given);
        if (kTop) {
            // thread t ranks key t % n of block t / n among all blocks' best
            const int n = a.n_top, total = a.split * n;
            uint64_t key = 0;
            if (t < total) {
                const uint32_t mine = map_to_rank(smem_u32(&s.f.best[t % n]), t / n);
                key = static_cast<uint64_t>(static_cast<uint32_t>(ld_cluster_s32(mine + 4))) << 32 |
                      static_cast<uint32_t>(ld_cluster_s32(mine));
                s.keys[t] = key;
            }
            // beams, whose rows may have fewer candidates: the places behind them are empty
            if (kBeam && a.split > 1) {
                const int filled = __syncthreads_count(key != 0);
                if (t >= filled && t < n) res.write_top(a, r, t, 0);
            } else if (a.split > 1) {
                __syncthreads();
            }
            // (a row has n keys, unless it is shorter: then there is no split, and the places behind stay empty)
            const int at = a.split == 1 ? t : rank_in<1>(s.keys, total, key, 0);
            if (t < total && at < n && (key || a.split == 1)) res.write_top(a, r, at, key);
        }
    }
    if (a.split > 1) cluster_sync_all();   // a block's shared memory stays until it has been read
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ..: kReaders threads read them one after the other, kFinishers threads
// finish each behind them.
template <class T, bool kBeam>
__global__ void __launch_bounds__(kReaders + kFinishers, kStreamBlocks) token_logprobs_stream_kernel(const LogprobArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    StreamShared<T>& s = *reinterpret_cast<StreamShared<T>*>(smem);
    constexpr int kAll = kReaders + kFinishers;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int buffer = 0;
    if (warp < kReaders / 32) {
        const int t = threadIdx.x;
        long long handed = 0;
        for (long long r = blockIdx.x; r < a.rows; r += gridDim.x, buffer ^= 1, ++handed) {
            const Row<T> row(a.logits, a.row_stride, r, a.vocab);
            const int batches = (row.pieces + kReaders * kBatch - 1) / (kReaders * kBatch);
            const int per_group = per_maximum<kReaders>(batches);
            if (handed >= 2) bar_sync(kBarEmpty + buffer, kAll);
            Stats st = read_pieces<T, true, kReaders>(row, 0, row.pieces, t, batches, per_group,
                                                         s.top[buffer] + maximum_place<T, kFinishers, kReaders>(t));
            if (const int edge = row.edge(t, a.vocab); edge >= 0) {
                const float x = static_cast<float>(row.x[edge]);
                st.raise(fmaxf(st.m, x));
                st.add(x);
            }
            st.join_warp();
            if (lane == 0) s.stats[buffer][warp] = st;
            bar_arrive(kBarFull + buffer, kAll);
        }
    } else {
        const int t = threadIdx.x - kReaders;
        for (long long r = blockIdx.x; r < a.rows; r += gridDim.x, buffer ^= 1) {
            const Row<T> row(a.logits, a.row_stride, r, a.vocab);
            const int batches = (row.pieces + kReaders * kBatch - 1) / (kReaders * kBatch);
            const int per_group = per_maximum<kReaders>(batches);
            const int groups = per_group ? (batches + per_group - 1) / per_group : 0;
            const int edge = row.edge(t, a.vocab);
            const float edge_value = edge >= 0 ? static_cast<float>(row.x[edge]) : -INFINITY;
            const int token = a.logprob ? given_token(a, r) : -1;
            const float given = token >= 0 ? static_cast<float>(row.x[token]) : 0.0f;
            bar_sync(kBarFull + buffer, kAll);
            find_best<T, kFinishers, kReaders, kBeam>(s.f, s.top[buffer], s.keys, row, a.n_top, 0, row.pieces, per_group, groups, t, edge, edge_value);
            sync_finders<kFinishers>();
            if (t < 32) {
                Stats all = lane < kReaders / 32 ? s.stats[buffer][lane] : Stats{-INFINITY, 0.0f, 0.0f};
                all.join_warp();
                const Result<kBeam> res(all);
                if (t == 0) res.write(a, r, all, token, given);
                if (t < a.n_top) res.write_top(a, r, t, s.f.best[t]);
            }
            sync_finders<kFinishers>();   // s.f is free for the next row
            if (r + 2 * static_cast<long long>(gridDim.x) < a.rows) bar_arrive(kBarEmpty + buffer, kAll);
        }
    }
}

// dx_i = g (1[i = token] - p_i) - h p_i (ln p_i + H) = g 1[i = token] - p_i (g + h (z_i + H)), z = x - lse.
// One block per run of 4 pieces a thread; dst has the logits' alignment or is written value by value.
template <class T>
__global__ void __launch_bounds__(kThreads) token_logprobs_backward_kernel(const LogprobGradArgs a)
{
    constexpr int kN = Piece<T>::kN;
    const long long r = blockIdx.x / static_cast<unsigned>(a.runs);
    const int run = static_cast<int>(blockIdx.x - r * a.runs);
    const Row<T> row(a.logits, a.row_stride, r, a.vocab);
    T* dx = static_cast<T*>(a.dlogits) + r * a.drow_stride;
    const bool vector = (reinterpret_cast<uintptr_t>(dx + row.head) & 15) == 0;
    uint4 v[kBatch];
    const int threads = blockDim.x, p0 = run * threads * kBatch + threadIdx.x;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
        if (p0 + j * threads < row.pieces) v[j] = row.body[p0 + j * threads];
    int token = a.token ? a.token[r] : -1;
    if (token >= a.vocab) {
        if (run == 0 && threadIdx.x == 0) record_error(a.status, MOE_ERR_INDEX);
        token = -1;
    }
    const float lse = a.lse[r], H = a.entropy ? a.entropy[r] : 0.0f;
    const bool none = lse == -INFINITY;   // nothing live in the row: no probability to move
    const float g = token >= 0 && a.dlogprob ? a.dlogprob[r] : 0.0f, h = a.dentropy ? a.dentropy[r] : 0.0f;
    const float gh = fmaf(h, H, g);
    auto grad = [&](float x) {
        const float z = max_nan(x - lse, -1e4f);   // p = 0 below; -inf would make NaN of 0 * z
        return none ? 0.0f : -exp2_fast(z * kLog2e) * fmaf(h, z, gh);
    };
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
        const int p = p0 + j * threads;
        if (p >= row.pieces) break;
        float x[kN];
        Piece<T>::unpack(v[j], x);
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = grad(x[i]);
        const int first = row.head + p * kN;
        if (token >= first && token < first + kN && !none) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if (first + i == token) x[i] += g;
        }
        if (vector) {
            *reinterpret_cast<uint4*>(dx + first) = Piece<T>::pack(x);
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) dx[first + i] = static_cast<T>(x[i]);
        }
    }
    if (run == 0) {
        const int i = row.edge(threadIdx.x, a.vocab);
        if (i >= 0) {
            const float x = grad(static_cast<float>(row.x[i]));
            dx[i] = static_cast<T>(i == token && !none ? x + g : x);
        }
    }
}

// Rows to blocks of NT threads, or to clusters of a.split of them.
template <int NT>
cudaError_t launch_rows(const LogprobArgs& a, cudaStream_t s)
{
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(static_cast<unsigned>(a.rows * a.split));
    c.blockDim = dim3(NT);
    c.dynamicSmemBytes = a.n_top == 0 ? offsetof(Shared<float>, f) : (a.bf16 ? sizeof(Shared<__nv_bfloat16>) : sizeof(Shared<float>));
    c.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(a.split);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    c.attrs = &attr;
    c.numAttrs = a.split > 1 ? 1 : 0;
    using B = __nv_bfloat16;
    if (a.stats) return cudaLaunchKernelEx(&c, a.bf16 ? token_logprobs_kernel<B, true, NT, true> : token_logprobs_kernel<float, true, NT, true>, a);
    const auto kernel = a.bf16 ? (a.n_top > 0 ? token_logprobs_kernel<B, true, NT, false> : token_logprobs_kernel<B, false, NT, false>)
                               : (a.n_top > 0 ? token_logprobs_kernel<float, true, NT, false> : token_logprobs_kernel<float, false, NT, false>);
    return cudaLaunchKernelEx(&c, kernel, a);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& args, cudaStream_t s)
{
    if (args.rows <= 0) return cudaSuccess;
    LogprobArgs a = args;
    // Few rows: a cluster of blocks per row, while a block keeps 8 pieces per thread and the rows' blocks are at most two
    // an SM.  Long rows gain (us for the 20 best of bf16 rows, with 1 / 2 / 4 / 8 blocks a row: one row of 131072 14.1 /
    // 10.3 / 8.8 / 8.7, 128 rows 20.4 / 15.4 / 16.4 / 25.7); short ones and many rows lose or stay (one row of 32000 7.8 / 8.2
    // / 7.7 / 7.9, 256 rows 10.3 / 13.7 / 20.9 / 40.8; of 131072 24.2 / 21.7 / 29.7 / 48.1).
    const long long pieces = static_cast<long long>(a.vocab) * (a.bf16 ? 2 : 4) / 16;
    a.split = 1;
    while (a.split < 8 && a.rows * a.split <= num_sms() && pieces / (a.split * 2) >= 8 * kThreads) a.split *= 2;
    if (a.rows * a.split > 0x7fffffffLL) return cudaErrorInvalidValue;
    const bool many = a.rows > blocks_of(kThreads) * static_cast<long long>(num_sms());   // more rows than blocks fit at once
    // Many short rows: what a row waits for (its loads, its search) is long against its work, so as many as fit, two
    // warps each (us for the 20 best of 4096 bf16 rows, two warps and otherwise: of 4000 22.7 and 39.5, of 16000 42.7 and
    // 51.7, of 20000 53.7 and 54.2, of 32000 66.8 and 64.8, of 50257 109 and 81; statistics alone of 16000 29.4 and 36.6).
    if (many && pieces <= 2560) return launch_rows<kFewThreads>(a, s);
    // Many long ones: rows are read ahead of their alternatives (20 best of 131072 bf16: 760 rows 40.8 us, 46.3 streamed;
    // 800 rows 54.9 and 46.6; 4096 rows 192 and 179).
    if (a.n_top > 0 && many) {
        const unsigned grid = static_cast<unsigned>(kStreamBlocks * num_sms());
        using B = __nv_bfloat16;
        const auto kernel = a.bf16 ? (a.stats ? token_logprobs_stream_kernel<B, true> : token_logprobs_stream_kernel<B, false>)
                                   : (a.stats ? token_logprobs_stream_kernel<float, true> : token_logprobs_stream_kernel<float, false>);
        kernel<<<grid, kReaders + kFinishers, a.bf16 ? sizeof(StreamShared<B>) : sizeof(StreamShared<float>), s>>>(a);
        return cudaGetLastError();
    }
    // One or two long rows an SM: more loads in flight for each (20 best of 200 / 300 rows of 131072 fp32: 28.2 / 35.0 us,
    // 34.9 / 38.4 with 256 threads; of 65536 bf16, which gain nothing, 13.2 / 15.4 and 12.5 / 15.9).
    if (a.split == 1 && a.rows > num_sms() && a.rows <= 2LL * num_sms() && pieces >= 12288) return launch_rows<kMoreThreads>(a, s);
    return launch_rows<kThreads>(a, s);
}

cudaError_t launch_token_logprobs_backward(const LogprobGradArgs& args, cudaStream_t s)
{
    if (args.rows <= 0) return cudaSuccess;
    LogprobGradArgs a = args;
    const long long pieces = static_cast<long long>(a.vocab) * (a.bf16 ? 2 : 4) / 16;
    // Equal runs, and as many threads as a run has work for (128786 x 1300 fp32: 191 us, with 256 threads always 241;
    // 20000 x 8200 bf16, a piece more than 256 threads take: 95 and 104).
    a.runs = static_cast<int>(std::max<long long>((pieces + kThreads * kBatch - 1) / (kThreads * kBatch), 1));
    const int threads = static_cast<int>(std::max<long long>((pieces + 32LL * kBatch * a.runs - 1) / (32LL * kBatch * a.runs) * 32, 32));
    if (a.rows * a.runs > 0x7fffffffLL) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(a.rows * a.runs);
    if (a.bf16)
        token_logprobs_backward_kernel<__nv_bfloat16><<<grid, threads, 0, s>>>(a);
    else
        token_logprobs_backward_kernel<float><<<grid, threads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
