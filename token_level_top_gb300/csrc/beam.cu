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
//
// Reordering: beam w continues beam p = parent[w].  The full pages of p are shared
// (table entries only).  The page that fills next has to be a beam's own: the first
// child of p keeps p's, every other child gets the one of a beam that nobody
// continues -- there are as many -- and the cached rows of p's copied into it.  So a
// step in which every beam goes on moves no cache at all.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kSelectThreads = 256;
constexpr int kMaxCandidates = MOE_MAX_BEAMS * MOE_MAX_TOP;

__global__ void __launch_bounds__(kSelectThreads) beam_select_kernel(const BeamArgs a)
{
    __shared__ double s_total[kMaxCandidates];
    __shared__ int s_valid;
    const int W = a.beams, n = a.n, count = W * n;
    const long long b = blockIdx.x;
    if (threadIdx.x == 0) s_valid = 0;
    __syncthreads();
    int valid = 0;
    for (int i = threadIdx.x; i < count; i += kSelectThreads) {
        const int w = i / n;
        const long long row = b * W + w;
        const float x = a.top_x[row * n + (i - w * n)], score = a.scores[row];
        const float2 stat = a.stats[row];   // maximum, sum of e^(x - maximum)
        double total = -INFINITY;
        // a row with NaN or +inf has no log probabilities (recorded where it was read), one of -inf alone no candidates
        if (x > -INFINITY && score > -INFINITY && stat.y == stat.y)
            total = static_cast<double>(score) + ((static_cast<double>(x) - stat.x) - log(static_cast<double>(stat.y)));
        if (score != score) record_error(a.status, MOE_ERR_NONFINITE);
        s_total[i] = total;
        valid += total > -INFINITY;
    }
    if (valid) atomicAdd(&s_valid, valid);
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kSelectThreads) {
        const double total = s_total[i];
        if (!(total > -INFINITY)) continue;
        const int w = i / n;
        int rank = i - w * n;
        for (int o = 0; o < W && rank < n; ++o) {
            if (o == w) continue;
            // how many of beam o's come before: its totals fall; equal ones of a lower beam do
            int lo = 0, hi = n;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                const double t = s_total[o * n + mid];
                if (o < w ? t >= total : t > total)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            rank += lo;
        }
        if (rank >= n) continue;
        a.out_scores[b * n + rank] = static_cast<float>(total);
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

constexpr int kMoveThreads = 256, kMoveDepth = 4;   // 16-byte pieces that a thread has in flight

// Where the beams' filling pages come from, decided by the first 64 threads of a block.
struct Homes {
    int parent[MOE_MAX_BEAMS];     // checked; -1: none
    int home[MOE_MAX_BEAMS];       // the beam whose filling page this one gets
    unsigned first[2], free[2];    // bits: the first of its parent's children; beams that nobody continues
};

__device__ __forceinline__ int nth_bit(const unsigned (&m)[2], int n)
{
    const int low = __popc(m[0]);
    return n < low ? __fns(m[0], 0, n + 1) : 32 + __fns(m[1], 0, n - low + 1);
}

__device__ __forceinline__ void find_homes(const BeamMoveArgs& a, long long b, Homes& h)
{
    const int w = threadIdx.x, W = a.beams;
    if (w < MOE_MAX_BEAMS) {
        int p = -1;
        if (w < W) {
            p = a.parents[b * a.parent_stride + w];
            if (p >= W) {
                if (blockIdx.y == 0) record_error(a.status, MOE_ERR_INDEX);
                p = -1;
            }
        }
        h.parent[w] = p < 0 ? -1 : p;
    }
    __syncthreads();
    if (w < MOE_MAX_BEAMS) {
        const int p = h.parent[w];
        bool first = p >= 0, free = w < W;
        for (int o = 0; o < W; ++o) {
            const int q = h.parent[o];
            if (o < w && q == p) first = false;
            if (q == w) free = false;
        }
        const unsigned fb = __ballot_sync(0xffffffffu, first), eb = __ballot_sync(0xffffffffu, free);
        if ((w & 31) == 0) {
            h.first[w >> 5] = fb;
            h.free[w >> 5] = eb;
        }
    }
    __syncthreads();
    if (w < W) {
        // the n-th beam that is no first child takes the n-th page left over
        const unsigned below = w < 32 ? (1u << w) - 1u : 0xffffffffu, above = w < 32 ? 0u : (1u << (w - 32)) - 1u;
        const bool first = h.first[w >> 5] >> (w & 31) & 1u;
        h.home[w] = first ? h.parent[w] : nth_bit(h.free, __popc(~h.first[0] & below) + __popc(~h.first[1] & above));
    }
    __syncthreads();
}

// Block (x, y): beam x of the batch, part y of its table row and of the rows it gets.
__global__ void __launch_bounds__(kMoveThreads) beam_reorder_kernel(const BeamMoveArgs a)
{
    __shared__ Homes h;
    const int W = a.beams;
    const long long b = blockIdx.x / static_cast<unsigned>(W), row = blockIdx.x;
    const int w = static_cast<int>(row - b * W);
    find_homes(a, b, h);
    const long long most = static_cast<long long>(a.max_pages) * a.page_size;
    long long len = a.seq_len[b];
    if (len < 0 || len > most) {
        if (threadIdx.x == 0 && blockIdx.y == 0 && w == 0) record_error(a.status, MOE_ERR_INDEX);
        len = len < 0 ? 0 : most;
    }
    const int full = static_cast<int>(len / a.page_size), rest = static_cast<int>(len - static_cast<long long>(full) * a.page_size);
    const int p = h.parent[w], home = h.home[w];
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
    auto place = [&](int cell, long long token_step, long long head_step) {
        const int token = by_token ? cell % rest : cell / a.n_kv_heads, head = by_token ? cell / rest : cell % a.n_kv_heads;
        return token * token_step + head * head_step;
    };
    auto at = [&](int i, int page) {
        const bool v = i >= pieces;
        const int k = v ? i - pieces : i, cell = k / per;
        return static_cast<char*>(v ? a.v : a.k) + page * a.page_bytes + place(cell, a.token_bytes, a.head_bytes) + (k - cell * per) * 16;
    };
    const int step = gridDim.y * kMoveThreads;
    for (int i0 = blockIdx.y * kMoveThreads + threadIdx.x; i0 < 2 * pieces; i0 += kMoveDepth * step) {
        uint4 x[kMoveDepth];
#pragma unroll
        for (int d = 0; d < kMoveDepth; ++d)
            if (i0 + d * step < 2 * pieces) x[d] = *reinterpret_cast<const uint4*>(at(i0 + d * step, src));
#pragma unroll
        for (int d = 0; d < kMoveDepth; ++d)
            if (i0 + d * step < 2 * pieces) *reinterpret_cast<uint4*>(at(i0 + d * step, dst)) = x[d];
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
    beam_select_kernel<<<static_cast<unsigned>(a.seqs), kSelectThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_beam_reorder(const BeamMoveArgs& a, cudaStream_t s)
{
    if (a.seqs <= 0) return cudaSuccess;
    // parts of a beam: its threads move kMoveDepth pieces twice each when its page is full
    const long long pieces = 2LL * a.page_size * a.n_kv_heads * (a.row_bytes / 16);
    const unsigned parts = static_cast<unsigned>(std::clamp<long long>(pieces / (2 * kMoveThreads * kMoveDepth), 1, 32));
    beam_reorder_kernel<<<dim3(static_cast<unsigned>(a.seqs) * a.beams, parts), kMoveThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
