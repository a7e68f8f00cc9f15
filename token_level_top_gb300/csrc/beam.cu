// beam.cu -- a step of beam search: the best continuations over all beams and the
// vocabulary, and the beams' page tables brought in line with the chosen parents.
//
// Selection: total(w, v) = score_w + x_wv - lse_w, the n largest of a sequence.  The
// logits are read once by the kernel of the token log probabilities, which leaves
// of every row the n largest values and the maximum and sum of its softmax; a second
// kernel, a block per sequence, ranks the beams' lists against each other.  A
// candidate's rank is its place in its own list plus, for every other beam, how many
// of that beam's come before it (a binary search: the lists are in order).  Totals
// are formed in fp64 from the value, the maximum and the logarithm of the sum: in
// fp32 two candidates a rounding apart (1e-6 at a total of 12) would change places.
// The sum itself is of fp32 terms in fp32, in an order that follows the row's 16-byte
// pieces; equal rows that start at other places of 16 bytes would have sums some 1e-7
// apart, and their candidates no ties.  So where rows start at several, the sums of
// beams that may be equal rows are taken again, by index (sum_by_index).
// Bounded by reading the logits: 64 x 8 rows of 131072 fp32 with the 16 best, one in
// twenty finished, 50 us of the 57 (268 MB: 0.80 of the copy rate).  A single search
// of 4 beams over 32000 tokens 12 us, two launches and the row's chain of searches.
//
// Reordering: beam w continues beam p = parent[w].  The full pages of p are shared
// (table entries only).  The page that fills next has to be a beam's own: the first
// child of p keeps p's, every other child gets the one of a beam that nobody
// continues -- there are as many -- and the cached rows of p's copied into it.  So a
// step in which every beam goes on moves no cache at all.  64 x 8 beams with a third
// to be moved (47 MB of rows both ways) 10.4 us; one search 3 us.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kSelectThreads = 256;
constexpr int kMaxCandidates = MOE_MAX_BEAMS * MOE_MAX_TOP;

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A double's bits as an integer of the same order (-0 comes below 0; there is none here).
__device__ __forceinline__ long long ordered(double x)
{
    const long long bits = __double_as_longlong(x);
    return bits ^ (bits >> 63 & 0x7fffffffffffffffLL);
}
constexpr long long kNoTotal = -0x7ff0000000000001LL;   // of -inf

// A row's sum of e^(x - maximum), by threads that take every kSelectThreads-th value: the same bits for equal rows, wherever
// they start.  For all threads of the block.  (Rare, so loads of single values, 16 in flight a thread: 64 x 8 rows of 131071
// fp32, all of a sequence's equal, 386 us, all different 60, of 50257 bf16 84 and 23.)
template <class T>
__device__ __noinline__ float sum_by_index(const BeamArgs& a, long long row, float maximum, float* buf)
{
    const T* const x = static_cast<const T*>(a.logits) + row * a.row_stride;
    float l = 0.0f;
#pragma unroll 16
    for (unsigned i = threadIdx.x; i < static_cast<unsigned>(a.vocab); i += kSelectThreads)
        l += exp2_fast((static_cast<float>(x[i]) - maximum) * 1.4426950408889634f);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = l;
    __syncthreads();
    l = buf[0];
    for (int i = 1; i < kSelectThreads / 32; ++i) l += buf[i];
    __syncthreads();
    return l;
}

// (Few fp64 operations: the chip does two a cycle and SM.  A logarithm a row instead of one a candidate, and ranking by integers:
// 60.1 to 57.4 us for 64 x 8 beams with 16 candidates, the logits read in 50.  Looking for equal rows only where they start
// apart, in an instance of its own: 0.4 us of 12.2 and 1 of 57.2.)
template <bool kApart>
__global__ void __launch_bounds__(kSelectThreads) beam_select_kernel(const BeamArgs a)
{
    __shared__ long long s_total[kMaxCandidates];
    __shared__ double s_log[MOE_MAX_BEAMS];
    __shared__ int s_valid;
    wait_for_previous();
    const int W = a.beams, n = a.n, count = W * n;
    const long long b = blockIdx.x;
    if (threadIdx.x == 0) s_valid = 0;
    if (threadIdx.x < W) {
        s_log[threadIdx.x] = log(static_cast<double>(a.stats[b * W + threadIdx.x].y));   // sum of e^(x - maximum)
        const float score = a.scores[b * W + threadIdx.x];
        if (score != score) record_error(a.status, MOE_ERR_NONFINITE);
    }
    __shared__ int s_again[kApart ? MOE_MAX_BEAMS : 1];
    __shared__ float s_buf[kApart ? kSelectThreads / 32 : 1];
    if (kApart && threadIdx.x < W) s_again[threadIdx.x] = 0;
    __syncthreads();
    if constexpr (kApart) {
        // beams that may be equal rows: the same best values, sums that differ, by no more than an order's roundings
        bool any = false;
        for (int i = threadIdx.x; i < W * W; i += kSelectThreads) {
            const int w = i / W, o = i - w * W;
            const float2 p = a.stats[b * W + w], q = a.stats[b * W + o];
            bool same = p.x == q.x && p.y != q.y && fabsf(p.y - q.y) <= 0x1p-10f * (p.y + q.y) && a.scores[b * W + w] > -INFINITY &&
                        a.scores[b * W + o] > -INFINITY;
            for (int j = 0; same && j < n; ++j) same = a.top_x[(b * W + w) * n + j] == a.top_x[(b * W + o) * n + j];
            if (same) s_again[w] = 1;
            any = any || same;
        }
        if (__syncthreads_or(any)) {
            for (int w = 0; w < W; ++w) {
                if (!s_again[w]) continue;
                const float maximum = a.stats[b * W + w].x;
                const float l = a.bf16 ? sum_by_index<__nv_bfloat16>(a, b * W + w, maximum, s_buf) : sum_by_index<float>(a, b * W + w, maximum, s_buf);
                if (threadIdx.x == 0) s_log[w] = log(static_cast<double>(l));
            }
            __syncthreads();
        }
    }
    int valid = 0;
    for (int i = threadIdx.x; i < count; i += kSelectThreads) {
        const int w = i / n;
        const long long row = b * W + w;
        const float x = a.top_x[row * n + (i - w * n)], score = a.scores[row];
        const float maximum = a.stats[row].x;
        const double log_sum = s_log[w];
        double total = -INFINITY;
        // a row with NaN or +inf has no log probabilities (recorded where it was read), one of -inf alone no candidates
        if (x > -INFINITY && score > -INFINITY && log_sum == log_sum)
            total = static_cast<double>(score) + ((static_cast<double>(x) - maximum) - log_sum) + 0.0;
        const long long key = total > -INFINITY ? ordered(total) : kNoTotal;
        s_total[i] = key;
        valid += key != kNoTotal;
    }
    if (valid) atomicAdd(&s_valid, valid);
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kSelectThreads) {
        const long long total = s_total[i];
        if (total == kNoTotal) continue;
        const int w = i / n;
        int rank = i - w * n;
        for (int o = 0; o < W && rank < n; ++o) {
            if (o == w) continue;
            // how many of beam o's come before: its totals fall; equal ones of a lower beam do
            int lo = 0, hi = n;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                const long long t = s_total[o * n + mid];
                if (o < w ? t >= total : t > total)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            rank += lo;
        }
        if (rank >= n) continue;
        a.out_scores[b * n + rank] = static_cast<float>(__longlong_as_double(total ^ (total >> 63 & 0x7fffffffffffffffLL)));
        a.parents[b * n + rank] = w;
        a.tokens[b * n + rank] = a.top_ids[b * count + i];
    }
    for (int i = s_valid + threadIdx.x; i < n; i += kSelectThreads) {
        a.out_scores[b * n + i] = -INFINITY;
        a.parents[b * n + i] = -1;
        a.tokens[b * n + i] = -1;
    }
}

// ---------------------------------------------------------------- reordering

constexpr int kMoveThreads = 128, kMoveDepth = 4;   // 16-byte pieces that a thread has in flight

// Beam w's parent (-1: none) and the beam whose filling page it gets, found by each warp for itself: lane l looks after
// beams l and l + 32.
struct Home {
    int parent, home;
};

__device__ __forceinline__ int nth_bit(const unsigned (&m)[2], int n)
{
    const int low = __popc(m[0]);
    return n < low ? __fns(m[0], 0, n + 1) : 32 + __fns(m[1], 0, n - low + 1);
}

__device__ __forceinline__ Home find_home(const BeamMoveArgs& a, long long b, int w)
{
    const int lane = threadIdx.x & 31, W = a.beams;
    int p[2] = {-1, -1};
    bool bad = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int beam = lane + 32 * h;
        if (beam < W) p[h] = a.parents[b * a.parent_stride + beam];
        bad = bad || p[h] >= W;
        if (p[h] >= W || p[h] < 0) p[h] = -1;
    }
    if (bad && blockIdx.y == 0 && w == 0 && threadIdx.x < 32) record_error(a.status, MOE_ERR_INDEX);
    // bits: the first of its parent's children; beams that somebody goes on from
    unsigned first[2] = {0, 0}, taken[2] = {0, 0};
    const unsigned same0 = __match_any_sync(0xffffffffu, p[0]);
    first[0] = __ballot_sync(0xffffffffu, p[0] >= 0 && __ffs(same0) - 1 == lane);
    taken[0] = __reduce_or_sync(0xffffffffu, p[0] >= 0 && p[0] < 32 ? 1u << p[0] : 0u);
    if (W > 32) {
        const unsigned same1 = __match_any_sync(0xffffffffu, p[1]);
        taken[1] = __reduce_or_sync(0xffffffffu, p[0] >= 32 ? 1u << (p[0] - 32) : 0u);
        // (p[1] is no first child if the lower beams have its parent)
        const unsigned low = p[1] < 0 ? 0u : (p[1] < 32 ? taken[0] >> p[1] : taken[1] >> (p[1] - 32)) & 1u;
        first[1] = __ballot_sync(0xffffffffu, p[1] >= 0 && !low && __ffs(same1) - 1 == lane);
        taken[0] |= __reduce_or_sync(0xffffffffu, p[1] >= 0 && p[1] < 32 ? 1u << p[1] : 0u);
        taken[1] |= __reduce_or_sync(0xffffffffu, p[1] >= 32 ? 1u << (p[1] - 32) : 0u);
    }
    const unsigned free[2] = {~taken[0] & (W >= 32 ? 0xffffffffu : (1u << W) - 1u),
                              W > 32 ? ~taken[1] & (W >= 64 ? 0xffffffffu : (1u << (W - 32)) - 1u) : 0u};
    Home h;
    h.parent = __shfl_sync(0xffffffffu, w < 32 ? p[0] : p[1], w & 31);
    // the n-th beam that is no first child takes the n-th page left over
    const unsigned below = w < 32 ? (1u << w) - 1u : 0xffffffffu, above = w < 32 ? 0u : (1u << (w - 32)) - 1u;
    const bool is_first = (w < 32 ? first[0] >> w : first[1] >> (w - 32)) & 1u;
    h.home = is_first ? h.parent : nth_bit(free, __popc(~first[0] & below) + __popc(~first[1] & above));
    return h;
}

// Block (x, y): beam x of the batch, part y of its table row and of the rows it gets.
__global__ void __launch_bounds__(kMoveThreads) beam_reorder_kernel(const BeamMoveArgs a)
{
    wait_for_previous();
    const int W = a.beams;
    const long long b = blockIdx.x / static_cast<unsigned>(W), row = blockIdx.x;
    const int w = static_cast<int>(row - b * W);
    const Home h = find_home(a, b, w);
    const long long most = static_cast<long long>(a.max_pages) * a.page_size;
    long long len = a.seq_len[b];
    if (len < 0 || len > most) {
        if (threadIdx.x == 0 && blockIdx.y == 0 && w == 0) record_error(a.status, MOE_ERR_INDEX);
        len = len < 0 ? 0 : most;
    }
    const int full = static_cast<int>(len / a.page_size), rest = static_cast<int>(len - static_cast<long long>(full) * a.page_size);
    const int p = h.parent, home = h.home;
    const int32_t* const mine = a.table + row * a.table_stride;
    const int32_t* const parent = a.table + (b * W + (p < 0 ? w : p)) * a.table_stride;
    const int32_t* const kept = a.table + (b * W + home) * a.table_stride;
    int32_t* const out = a.table_out + row * a.table_out_stride;
    for (int j = blockIdx.y * kMoveThreads + threadIdx.x; j < a.max_pages; j += gridDim.y * kMoveThreads)
        out[j] = j < full ? parent[j] : (j == full && rest > 0 ? kept[j] : mine[j]);

    if (rest == 0 || p < 0 || home == p) return;
    const int src = parent[full], dst = kept[full];
    if (src < 0 || src >= a.n_pages || dst < 0 || dst >= a.n_pages) {
        if (threadIdx.x == 0 && blockIdx.y == 0) record_error(a.status, MOE_ERR_INDEX);
        return;
    }
    if (src == dst) return;
    const int cells = rest * a.n_kv_heads, per = a.row_bytes / 16, pieces = cells * per;   // of the keys; the values' behind them
    // the place of a (token, head) cell in a page: the nearer one runs fastest
    const bool by_token = a.head_bytes > a.token_bytes;
    const int run = by_token ? rest : a.n_kv_heads;
    const float inverse = 1.0f / static_cast<float>(run);
    auto place = [&](int cell, long long token_step, long long head_step) {
        // (a division by the reciprocal is off by one at most below 2^22)
        int q = cells < 1 << 22 ? static_cast<int>(static_cast<float>(cell) * inverse) : cell / run;
        int left = cell - q * run;
        if (left < 0) --q, left += run;
        if (left >= run) ++q, left -= run;
        return by_token ? left * token_step + q * head_step : q * token_step + left * head_step;
    };
    const int shift = 31 - __clz(per);
    auto at = [&](int i) {
        const bool v = i >= pieces;
        const int k = v ? i - pieces : i, cell = k >> shift;
        return static_cast<char*>(v ? a.v : a.k) + place(cell, a.token_bytes, a.head_bytes) + (k - (cell << shift)) * 16;
    };
    const long long from = src * a.page_bytes, to = dst * a.page_bytes;
    const int step = gridDim.y * kMoveThreads;
    for (int i0 = blockIdx.y * kMoveThreads + threadIdx.x; i0 < 2 * pieces; i0 += kMoveDepth * step) {
        uint4 x[kMoveDepth];
        char* p[kMoveDepth];
#pragma unroll
        for (int d = 0; d < kMoveDepth; ++d)
            if (i0 + d * step < 2 * pieces) {
                p[d] = at(i0 + d * step);
                x[d] = *reinterpret_cast<const uint4*>(p[d] + from);
            }
#pragma unroll
        for (int d = 0; d < kMoveDepth; ++d)
            if (i0 + d * step < 2 * pieces) *reinterpret_cast<uint4*>(p[d] + to) = x[d];
    }
    if (!a.k_exp) return;
    for (int i = blockIdx.y * kMoveThreads + threadIdx.x; i < 2 * cells; i += step) {
        uint8_t* const e = i < cells ? a.k_exp : a.v_exp;
        const long long cell = place(i < cells ? i : i - cells, a.exp_token_stride, a.exp_head_stride);
        e[dst * a.exp_page_stride + cell] = e[src * a.exp_page_stride + cell];
    }
}

}  // namespace

size_t beam_ws_bytes(long long rows, int n, BeamWorkspace* at)
{
    if (rows < 0 || rows > 0x7fffffffLL || n < 1 || n > MOE_MAX_TOP) return 0;
    const size_t r = static_cast<size_t>(rows), up = 255;
    BeamWorkspace w;
    w.stats = kBeamCtrlBytes;
    w.ids = w.stats + ((r * sizeof(float2) + up) & ~up);
    w.x = w.ids + ((r * n * 4 + up) & ~up);
    if (at) *at = w;
    return w.x + ((r * n * 4 + up) & ~up);
}

cudaError_t launch_beam_select(const BeamArgs& a, cudaStream_t s)
{
    if (a.seqs <= 0) return cudaSuccess;
    LogprobArgs l{};
    l.rows = static_cast<long long>(a.seqs) * a.beams;
    l.vocab = a.vocab;
    l.bf16 = a.bf16;
    l.logits = a.logits;
    l.row_stride = a.row_stride;
    l.n_top = a.n;
    l.stats = a.stats;
    l.top_ids = a.top_ids;
    l.top_logprobs = a.top_x;
    l.status = a.status;
    const cudaError_t e = launch_token_logprobs(l, s);
    if (e != cudaSuccess) return e;
    return launch_after(a.apart ? beam_select_kernel<true> : beam_select_kernel<false>, dim3(static_cast<unsigned>(a.seqs)), kSelectThreads, 0, s, a);
}

cudaError_t launch_beam_reorder(const BeamMoveArgs& a, cudaStream_t s)
{
    if (a.seqs <= 0) return cudaSuccess;
    // Parts of a beam: when its page is full a thread moves kMoveDepth pieces four times, or once while that fills the GPU.  What
    // it takes is mostly the chain parent -> tables -> pages -> rows, so short blocks, many to an SM (64 x 8 beams, pages of
    // 64 rows of 8 heads of 128, a third of the beams moved: 10.2 us; 256 threads with 8 pieces twice 12.4, once 16.6).
    const long long pieces = 2LL * a.page_size * a.n_kv_heads * (a.row_bytes / 16), beams = static_cast<long long>(a.seqs) * a.beams;
    const long long once = (pieces + kMoveThreads * kMoveDepth - 1) / (kMoveThreads * kMoveDepth);
    const unsigned parts = static_cast<unsigned>(std::clamp<long long>(beams * once <= 8LL * num_sms() ? once : (once + 3) / 4, 1, 32));
    return launch_after(beam_reorder_kernel, dim3(static_cast<unsigned>(beams), parts), kMoveThreads, 0, s, a);
}

}  // namespace moe
