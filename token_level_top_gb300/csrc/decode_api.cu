// decode_api.cu -- the C ABI around the layer: argument checks for the paged
// cache, the attentions over it, the log probabilities, beam search and the norm.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kMaxHeads = 1024;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

moe_status_t check_cache(const moe_kv_cache_t* c)
{
    if (!c || !c->k || !c->v || c->type > MOE_KV_E4M3) return MOE_ERR_INVALID_ARG;
    if (c->n_pages <= 0 || c->page_size <= 0 || c->n_kv_heads <= 0) return MOE_ERR_INVALID_ARG;
    const bool e4m3 = c->type == MOE_KV_E4M3;
    if ((c->k_exp != nullptr) != e4m3 || (c->v_exp != nullptr) != e4m3) return MOE_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ERR_UNSUPPORTED;
    if (c->n_kv_heads > kMaxHeads || c->page_stride < 0 || c->token_stride < 0) return MOE_ERR_UNSUPPORTED;
    const int64_t unit = e4m3 ? 16 : 8;   // elements per 16 bytes
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % unit || c->token_stride % unit ||
        c->head_stride % unit)
        return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

moe_status_t append(const moe_kv_cache_t* c, const moe_append_t* p, const moe_rotation_t* r, int32_t* status, void* stream)
{
    moe_status_t st = check_cache(c);
    if (st != MOE_OK) return st;
    if (!p || p->T < 0 || p->n_seqs < 0 || p->max_pages < 0 || p->n_heads < 0 || p->table_stride < 0 || (p->flags & ~MOE_ROTATE_INTERLEAVED) != 0)
        return MOE_ERR_INVALID_ARG;
    if (p->rot_dim < 0 || p->rot_dim > c->head_dim || p->rot_dim % 16 != 0 || p->n_heads > kMaxHeads)
        return MOE_ERR_UNSUPPORTED;
    if (r && (r->n_axes <= 0 || r->axis_stride < 0)) return MOE_ERR_INVALID_ARG;
    if (r && r->n_axes > MOE_MAX_AXES) return MOE_ERR_UNSUPPORTED;
    if (p->T == 0) return MOE_OK;
    if (r && (!r->rotary || p->rot_dim == 0)) return MOE_ERR_INVALID_ARG;
    if (p->max_pages == 0 || !p->pos || !p->page_table || !p->k || !p->v || (p->rot_dim > 0 && !p->phase)) return MOE_ERR_INVALID_ARG;
    if ((p->n_heads > 0) != (p->q != nullptr) || (p->n_heads > 0) != (p->q_out != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!p->seq && p->T > p->n_seqs) return MOE_ERR_INVALID_ARG;
    const int64_t strides[] = {p->q_token_stride, p->q_head_stride, p->k_token_stride,     p->k_head_stride,
                               p->v_token_stride, p->v_head_stride, p->q_out_token_stride, p->q_out_head_stride};
    for (int64_t s : strides)
        if (s % 8) return MOE_ERR_MISALIGNED;
    for (int64_t s : {p->q_head_stride, p->k_head_stride, p->v_head_stride, p->q_out_head_stride, 2 * c->head_stride})
        if (s > INT32_MAX || s < INT32_MIN) return MOE_ERR_UNSUPPORTED;   // the kernel holds them in 32 bits
    if (!aligned(p->q, 16) || !aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->q_out, 16) || !aligned(p->phase, 16))
        return MOE_ERR_MISALIGNED;
    AppendArgs a{};
    a.T = p->T;
    a.n_seqs = p->n_seqs;
    a.max_pages = p->max_pages;
    a.n_heads = p->n_heads;
    a.n_kv_heads = c->n_kv_heads;
    a.rot_dim = p->rot_dim;
    a.n_pages = c->n_pages;
    a.page_size = c->page_size;
    a.interleaved = (p->flags & MOE_ROTATE_INTERLEAVED) != 0;
    a.pos = p->pos;
    a.seq = p->seq;
    a.page_table = p->page_table;
    a.table_stride = p->table_stride;
    a.phase = p->phase;
    a.q = static_cast<const __nv_bfloat16*>(p->q);
    a.k = static_cast<const __nv_bfloat16*>(p->k);
    a.v = static_cast<const __nv_bfloat16*>(p->v);
    a.q_out = static_cast<__nv_bfloat16*>(p->q_out);
    a.q_token_stride = p->q_token_stride;
    a.k_token_stride = p->k_token_stride;
    a.v_token_stride = p->v_token_stride;
    a.q_out_token_stride = p->q_out_token_stride;
    a.q_head = static_cast<int>(p->q_head_stride);
    a.k_head = static_cast<int>(p->k_head_stride);
    a.v_head = static_cast<int>(p->v_head_stride);
    a.q_out_head = static_cast<int>(p->q_out_head_stride);
    a.cache_head = static_cast<int>(c->head_stride * (c->type == MOE_KV_E4M3 ? 1 : 2));
    a.cache_k = c->k;
    a.cache_v = c->v;
    a.k_exp = static_cast<uint8_t*>(c->k_exp);
    a.v_exp = static_cast<uint8_t*>(c->v_exp);
    a.page_stride = c->page_stride;
    a.token_stride = c->token_stride;
    a.exp_page_stride = c->exp_page_stride;
    a.exp_token_stride = c->exp_token_stride;
    a.exp_head_stride = c->exp_head_stride;
    a.status = status;
    if (r) {
        a.rotary = r->rotary;
        a.axis = r->axis;
        a.axis_stride = r->axis_stride;
        a.n_axes = r->n_axes;
    }
    return cuda_status(
        launch_kv_append(a, c->head_dim, c->type == MOE_KV_E4M3, static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_rope_phase(int32_t n, const double* inv_freq, uint64_t* phase)
{
    if (n < 0 || (n > 0 && (!inv_freq || !phase))) return MOE_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i) {
        if (!isfinite(inv_freq[i])) return MOE_ERR_INVALID_ARG;
        const double turns = inv_freq[i] / 6.283185307179586;
        const double v = ldexp(turns - floor(turns), 64);
        phase[i] = v < 0x1p64 ? static_cast<uint64_t>(v) : 0;
    }
    return MOE_OK;
}

moe_status_t moe_kv_append(const moe_kv_cache_t* c, const moe_append_t* p, int32_t* status, void* stream)
{
    return append(c, p, nullptr, status, stream);
}

moe_status_t moe_kv_append_axes(const moe_kv_cache_t* c, const moe_append_t* p, const moe_rotation_t* r, int32_t* status,
                                void* stream)
{
    return r ? append(c, p, r, status, stream) : MOE_ERR_INVALID_ARG;
}

size_t moe_paged_attention_workspace_size(int32_t head_dim) { return paged_attention_ws_bytes(head_dim); }

moe_status_t moe_paged_attention_workspace_init(void* ws, size_t ws_bytes, void* stream)
{
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < kAttentionCtrlBytes) return MOE_ERR_WORKSPACE;
    return cuda_status(cudaMemsetAsync(ws, 0, kAttentionCtrlBytes, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_paged_attention(const moe_kv_cache_t* c, const moe_attention_t* p, void* ws, size_t ws_bytes,
                                 void* stream)
{
    moe_status_t st = check_cache(c);
    if (st != MOE_OK) return st;
    if (!p || p->B < 0 || p->n_heads <= 0 || p->n_heads % c->n_kv_heads != 0 || p->max_pages < 0 || p->window < 0 ||
        p->table_stride < 0 || !isfinite(p->scale))
        return MOE_ERR_INVALID_ARG;
    // the kernel's place of a row in a page is a 32-bit byte offset
    const int64_t elt = c->type == MOE_KV_E4M3 ? 1 : 2, far = int64_t{1} << 32;
    if (p->n_heads > kMaxHeads || c->page_stride >= far / elt || c->token_stride >= far / elt) return MOE_ERR_UNSUPPORTED;
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < paged_attention_ws_bytes(c->head_dim)) return MOE_ERR_WORKSPACE;
    if (p->B == 0) return MOE_OK;
    if (p->max_pages == 0 || !p->seq_len || !p->page_table || !p->q || !p->out) return MOE_ERR_INVALID_ARG;
    if (!aligned(p->q, 16) || !aligned(p->out, 16) || p->q_token_stride % 8 || p->q_head_stride % 8 ||
        p->out_token_stride % 8 || p->out_head_stride % 8)
        return MOE_ERR_MISALIGNED;
    AttentionArgs a{};
    a.B = p->B;
    a.n_heads = p->n_heads;
    a.n_kv_heads = c->n_kv_heads;
    a.max_pages = p->max_pages;
    a.window = p->window;
    a.n_pages = c->n_pages;
    a.page_size = c->page_size;
    a.scale = p->scale;
    a.seq_len = p->seq_len;
    a.page_table = p->page_table;
    a.table_stride = p->table_stride;
    a.q = static_cast<const __nv_bfloat16*>(p->q);
    a.out = static_cast<__nv_bfloat16*>(p->out);
    a.lse = p->lse;
    a.q_token_stride = p->q_token_stride;
    a.q_head_stride = p->q_head_stride;
    a.out_token_stride = p->out_token_stride;
    a.out_head_stride = p->out_head_stride;
    a.k = c->k;
    a.v = c->v;
    a.k_exp = static_cast<const uint8_t*>(c->k_exp);
    a.v_exp = static_cast<const uint8_t*>(c->v_exp);
    a.page_stride = c->page_stride;
    a.token_stride = c->token_stride;
    a.head_stride = c->head_stride;
    a.exp_page_stride = c->exp_page_stride;
    a.exp_token_stride = c->exp_token_stride;
    a.exp_head_stride = c->exp_head_stride;
    a.ws = ws;
    a.status = static_cast<int*>(ws);
    return cuda_status(
        launch_paged_attention(a, c->head_dim, c->type == MOE_KV_E4M3, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_token_logprobs(int64_t rows, int32_t vocab, uint32_t type, const void* logits, int64_t row_stride,
                                const int32_t* token, int32_t n_top, float* logprob, float* entropy, float* lse,
                                int32_t* top_ids, float* top_logprobs, int32_t* status, void* stream)
{
    if (rows < 0 || vocab <= 0 || type > MOE_LOGITS_BF16 || row_stride < 0 || n_top < 0) return MOE_ERR_INVALID_ARG;
    if (n_top > MOE_MAX_TOP || rows > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!logits || (logprob && !token) || (n_top > 0 && (!top_ids || !top_logprobs))) return MOE_ERR_INVALID_ARG;
    if (!aligned(logits, type == MOE_LOGITS_BF16 ? 2 : 4)) return MOE_ERR_MISALIGNED;
    LogprobArgs a{};
    a.rows = rows;
    a.vocab = vocab;
    a.bf16 = type == MOE_LOGITS_BF16;
    a.logits = logits;
    a.row_stride = row_stride;
    a.token = token;
    a.n_top = n_top;
    a.logprob = logprob;
    a.entropy = entropy;
    a.lse = lse;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.status = status;
    return cuda_status(launch_token_logprobs(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_token_logprobs_backward(int64_t rows, int32_t vocab, uint32_t type, const void* logits,
                                         int64_t row_stride, const int32_t* token, const float* lse,
                                         const float* entropy, const float* dlogprob, const float* dentropy,
                                         void* dlogits, int64_t drow_stride, int32_t* status, void* stream)
{
    if (rows < 0 || vocab <= 0 || type > MOE_LOGITS_BF16 || row_stride < 0 || (rows > 1 && drow_stride < vocab))
        return MOE_ERR_INVALID_ARG;
    if (rows > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!logits || !lse || !dlogits || (dentropy && !entropy) || (dlogprob && !token)) return MOE_ERR_INVALID_ARG;
    const size_t elt = type == MOE_LOGITS_BF16 ? 2 : 4;
    if (!aligned(logits, elt) || !aligned(dlogits, elt)) return MOE_ERR_MISALIGNED;
    if (logits == dlogits && rows > 1 && row_stride != drow_stride) return MOE_ERR_INVALID_ARG;
    LogprobGradArgs a{};
    a.rows = rows;
    a.vocab = vocab;
    a.bf16 = type == MOE_LOGITS_BF16;
    a.logits = logits;
    a.row_stride = row_stride;
    a.token = token;
    a.lse = lse;
    a.entropy = entropy;
    a.dlogprob = dlogprob;
    a.dentropy = dentropy;
    a.dlogits = dlogits;
    a.drow_stride = drow_stride;
    a.status = status;
    return cuda_status(launch_token_logprobs_backward(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_tree_attention_workspace_size(int32_t head_dim) { return tree_attention_ws_bytes(head_dim); }

moe_status_t moe_tree_attention_workspace_init(void* ws, size_t ws_bytes, void* stream)
{
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < kTreeCtrlBytes) return MOE_ERR_WORKSPACE;
    return cuda_status(cudaMemsetAsync(ws, 0, kTreeCtrlBytes, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_tree_attention(const moe_kv_cache_t* c, const moe_tree_attention_t* p, void* ws, size_t ws_bytes,
                                void* stream)
{
    moe_status_t st = check_cache(c);
    if (st != MOE_OK) return st;
    if (!p || p->B < 0 || p->T < 0 || p->n_heads <= 0 || p->n_heads % c->n_kv_heads != 0 || p->max_pages < 0 || p->window < 0 ||
        p->table_stride < 0 || !isfinite(p->scale))
        return MOE_ERR_INVALID_ARG;
    if (p->n_heads > kMaxHeads) return MOE_ERR_UNSUPPORTED;
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < tree_attention_ws_bytes(c->head_dim)) return MOE_ERR_WORKSPACE;
    if (p->B == 0 || p->T == 0) return MOE_OK;
    if (p->max_pages == 0 || !p->row_start || !p->seq_len || !p->page_table || !p->q || !p->out) return MOE_ERR_INVALID_ARG;
    if (!aligned(p->q, 16) || !aligned(p->out, 16) || p->q_token_stride % 8 || p->q_head_stride % 8 ||
        p->out_token_stride % 8 || p->out_head_stride % 8)
        return MOE_ERR_MISALIGNED;
    TreeArgs a{};
    a.B = p->B;
    a.T = p->T;
    a.n_heads = p->n_heads;
    a.n_kv_heads = c->n_kv_heads;
    a.max_pages = p->max_pages;
    a.window = p->window;
    a.n_pages = c->n_pages;
    a.page_size = c->page_size;
    a.scale = p->scale;
    a.row_start = p->row_start;
    a.seq_len = p->seq_len;
    a.mask = p->mask;
    a.page_table = p->page_table;
    a.table_stride = p->table_stride;
    a.q = static_cast<const __nv_bfloat16*>(p->q);
    a.out = static_cast<__nv_bfloat16*>(p->out);
    a.lse = p->lse;
    a.q_token_stride = p->q_token_stride;
    a.q_head_stride = p->q_head_stride;
    a.out_token_stride = p->out_token_stride;
    a.out_head_stride = p->out_head_stride;
    const int64_t elt = c->type == MOE_KV_E4M3 ? 1 : 2;
    a.k = static_cast<const char*>(c->k);
    a.v = static_cast<const char*>(c->v);
    a.k_exp = static_cast<const uint8_t*>(c->k_exp);
    a.v_exp = static_cast<const uint8_t*>(c->v_exp);
    a.page_bytes = c->page_stride * elt;
    a.token_bytes = c->token_stride * elt;
    a.head_bytes = c->head_stride * elt;
    a.exp_page_stride = c->exp_page_stride;
    a.exp_token_stride = c->exp_token_stride;
    a.exp_head_stride = c->exp_head_stride;
    a.ws = ws;
    a.status = static_cast<int*>(ws);
    return cuda_status(launch_tree_attention(a, c->head_dim, c->type == MOE_KV_E4M3, static_cast<cudaStream_t>(stream)));
}

size_t moe_beam_workspace_size(int64_t rows, int32_t n) { return beam_ws_bytes(rows, n, nullptr); }

moe_status_t moe_beam_workspace_init(void* ws, size_t ws_bytes, void* stream)
{
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < kBeamCtrlBytes) return MOE_ERR_WORKSPACE;
    return cuda_status(cudaMemsetAsync(ws, 0, kBeamCtrlBytes, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_beam_select(int32_t seqs, int32_t beams, int32_t vocab, uint32_t type, const void* logits,
                             int64_t row_stride, const float* scores, int32_t n, float* out_scores, int32_t* parents,
                             int32_t* tokens, void* ws, size_t ws_bytes, void* stream)
{
    if (seqs < 0 || beams <= 0 || vocab <= 0 || n <= 0 || type > MOE_LOGITS_BF16 || row_stride < 0) return MOE_ERR_INVALID_ARG;
    if (n > MOE_MAX_TOP || beams > MOE_MAX_BEAMS || static_cast<int64_t>(seqs) * beams > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
    BeamWorkspace at;
    if (ws_bytes < beam_ws_bytes(static_cast<int64_t>(seqs) * beams, n, &at)) return MOE_ERR_WORKSPACE;
    if (seqs == 0) return MOE_OK;
    if (!logits || !scores || !out_scores || !parents || !tokens) return MOE_ERR_INVALID_ARG;
    if (!aligned(logits, type == MOE_LOGITS_BF16 ? 2 : 4)) return MOE_ERR_MISALIGNED;
    BeamArgs a{};
    a.seqs = seqs;
    a.beams = beams;
    a.vocab = vocab;
    a.n = n;
    a.bf16 = type == MOE_LOGITS_BF16;
    a.apart = beams > 1 && row_stride % (a.bf16 ? 8 : 4) != 0;
    a.logits = logits;
    a.row_stride = row_stride;
    a.scores = scores;
    a.out_scores = out_scores;
    a.parents = parents;
    a.tokens = tokens;
    a.stats = ws_at<float2>(ws, at.stats);
    a.top_ids = ws_at<int32_t>(ws, at.ids);
    a.top_x = ws_at<float>(ws, at.x);
    a.status = static_cast<int*>(ws);
    return cuda_status(launch_beam_select(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_beam_reorder(const moe_kv_cache_t* c, const moe_beam_reorder_t* p, int32_t* status, void* stream)
{
    moe_status_t st = check_cache(c);
    if (st != MOE_OK) return st;
    if (!p || p->seqs < 0 || p->beams <= 0 || p->max_pages < 0 || p->parent_stride < 0 || p->table_stride < 0)
        return MOE_ERR_INVALID_ARG;
    if (p->beams > MOE_MAX_BEAMS || static_cast<int64_t>(p->seqs) * p->beams > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
    if (p->seqs == 0 || p->max_pages == 0) return MOE_OK;
    if (!p->parents || !p->seq_len || !p->page_table || !p->page_table_out) return MOE_ERR_INVALID_ARG;
    const int64_t rows = static_cast<int64_t>(p->seqs) * p->beams;
    if (rows > 1 && p->table_out_stride < p->max_pages) return MOE_ERR_INVALID_ARG;
    // the tables may not overlap: a beam's new row is made of other beams' old ones
    const int32_t *in = p->page_table, *in_end = in + (rows - 1) * p->table_stride + p->max_pages;
    const int32_t *out = p->page_table_out, *out_end = out + (rows - 1) * p->table_out_stride + p->max_pages;
    if (in < out_end && out < in_end) return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(c->page_size) * c->n_kv_heads * (c->head_dim / 16) > 0x1fffffffLL) return MOE_ERR_UNSUPPORTED;
    const int64_t elt = c->type == MOE_KV_E4M3 ? 1 : 2;
    BeamMoveArgs a{};
    a.seqs = p->seqs;
    a.beams = p->beams;
    a.max_pages = p->max_pages;
    a.n_pages = c->n_pages;
    a.page_size = c->page_size;
    a.n_kv_heads = c->n_kv_heads;
    a.row_bytes = static_cast<int>(c->head_dim * elt);
    a.parents = p->parents;
    a.parent_stride = p->parent_stride;
    a.seq_len = p->seq_len;
    a.table = p->page_table;
    a.table_stride = p->table_stride;
    a.table_out = p->page_table_out;
    a.table_out_stride = p->table_out_stride;
    a.k = c->k;
    a.v = c->v;
    a.k_exp = static_cast<uint8_t*>(c->k_exp);
    a.v_exp = static_cast<uint8_t*>(c->v_exp);
    a.page_bytes = c->page_stride * elt;
    a.token_bytes = c->token_stride * elt;
    a.head_bytes = c->head_stride * elt;
    a.exp_page_stride = c->exp_page_stride;
    a.exp_token_stride = c->exp_token_stride;
    a.exp_head_stride = c->exp_head_stride;
    a.status = status;
    return cuda_status(launch_beam_reorder(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_rms_norm_workspace_size(int32_t cols) { return rms_norm_ws_bytes(cols); }

moe_status_t moe_rms_norm(const moe_rms_norm_t* p, int32_t* status, void* stream)
{
    if (!p || p->rows < 0 || p->cols <= 0 || p->type > MOE_ROWS_BF16 || p->weight_type > MOE_ROWS_BF16) return MOE_ERR_INVALID_ARG;
    if (!(p->eps >= 1e-30f) || !isfinite(p->eps)) return MOE_ERR_INVALID_ARG;
    if (p->cols > kMaxNormCols || p->rows > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
    if ((p->codes != nullptr) != (p->scales != nullptr) || (p->sum && (!p->residual || p->sum == p->y))) return MOE_ERR_INVALID_ARG;
    if (p->x_stride < 0 || (p->residual && p->residual_stride < 0)) return MOE_ERR_INVALID_ARG;
    if (p->rows > 1 && ((p->sum && p->sum_stride < p->cols) || (p->y && p->y_stride < p->cols) || (p->codes && p->codes_stride < p->cols)))
        return MOE_ERR_INVALID_ARG;
    if (p->rows == 0) return MOE_OK;
    if (!p->x || (!p->y && !p->codes && !p->sum)) return MOE_ERR_INVALID_ARG;
    const size_t elt = p->type == MOE_ROWS_BF16 ? 2 : 4;
    for (const void* t : {p->x, p->residual, static_cast<const void*>(p->sum), static_cast<const void*>(p->y)})
        if (!aligned(t, elt)) return MOE_ERR_MISALIGNED;
    if (!aligned(p->weight, p->weight_type == MOE_ROWS_BF16 ? 2 : 4) || !aligned(p->scales, 4)) return MOE_ERR_MISALIGNED;
    // a place that is read by one row's threads and written by another's: only whole rows may coincide
    const void* const ins[] = {p->x, p->residual};
    const int64_t in_strides[] = {p->x_stride, p->residual_stride};
    for (int i = 0; i < 2; ++i) {
        if (!ins[i] || p->rows == 1) continue;
        if ((ins[i] == p->sum && in_strides[i] != p->sum_stride) || (ins[i] == p->y && in_strides[i] != p->y_stride))
            return MOE_ERR_INVALID_ARG;
    }
    NormArgs a{};
    a.rows = p->rows;
    a.cols = p->cols;
    a.bf16 = p->type == MOE_ROWS_BF16;
    a.weight_f32 = p->weight_type == MOE_ROWS_F32;
    a.eps = p->eps;
    a.x = p->x;
    a.residual = p->residual;
    a.weight = p->weight;
    a.sum = p->sum;
    a.y = p->y;
    a.codes = static_cast<uint8_t*>(p->codes);
    a.scales = p->scales;
    a.x_stride = p->x_stride;
    a.residual_stride = p->residual ? p->residual_stride : 0;
    a.sum_stride = p->sum ? p->sum_stride : 0;
    a.y_stride = p->y ? p->y_stride : 0;
    a.codes_stride = p->codes ? p->codes_stride : 0;
    a.status = status;
    return cuda_status(launch_rms_norm(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_rms_norm_backward(const moe_rms_norm_grad_t* p, void* ws, size_t ws_bytes, void* stream)
{
    if (!p || p->rows < 0 || p->cols <= 0 || p->type > MOE_ROWS_BF16 || p->dy_type > MOE_ROWS_BF16 || p->weight_type > MOE_ROWS_BF16)
        return MOE_ERR_INVALID_ARG;
    if (!(p->eps >= 1e-30f) || !isfinite(p->eps)) return MOE_ERR_INVALID_ARG;
    if (p->cols > kMaxNormCols || (p->type == MOE_ROWS_F32 && p->dy_type != MOE_ROWS_F32)) return MOE_ERR_UNSUPPORTED;
    if (p->x_stride < 0 || p->dy_stride < 0 || (p->dsum && p->dsum_stride < 0) || (p->rows > 1 && p->dx_stride < p->cols))
        return MOE_ERR_INVALID_ARG;
    if (p->dweight) {
        if (!ws) return MOE_ERR_INVALID_ARG;
        if (!aligned(ws, 256) || !aligned(p->dweight, 4)) return MOE_ERR_MISALIGNED;
        if (ws_bytes < rms_norm_ws_bytes(p->cols)) return MOE_ERR_WORKSPACE;
    }
    if (p->rows > 0) {
        if (!p->x || !p->dy || !p->dx) return MOE_ERR_INVALID_ARG;
        const size_t elt = p->type == MOE_ROWS_BF16 ? 2 : 4;
        if (!aligned(p->x, elt) || !aligned(p->dsum, elt) || !aligned(p->dx, elt) ||
            !aligned(p->dy, p->dy_type == MOE_ROWS_BF16 ? 2 : 4) || !aligned(p->weight, p->weight_type == MOE_ROWS_BF16 ? 2 : 4))
            return MOE_ERR_MISALIGNED;
        if (p->rows > 1 && ((p->dx == p->x && p->dx_stride != p->x_stride) || (p->dx == p->dsum && p->dx_stride != p->dsum_stride) ||
                            (p->dx == p->dy && (p->dx_stride != p->dy_stride || p->dy_type != p->type))))
            return MOE_ERR_INVALID_ARG;
    }
    NormGradArgs a{};
    a.rows = p->rows;
    a.cols = p->cols;
    a.bf16 = p->type == MOE_ROWS_BF16;
    a.dy_f32 = p->dy_type == MOE_ROWS_F32;
    a.weight_f32 = p->weight_type == MOE_ROWS_F32;
    a.eps = p->eps;
    a.x = p->x;
    a.weight = p->weight;
    a.dy = p->dy;
    a.dsum = p->dsum;
    a.dx = p->dx;
    a.dweight = p->dweight;
    a.parts = p->dweight ? ws_at<float>(ws, 0) : nullptr;
    a.x_stride = p->x_stride;
    a.dy_stride = p->dy_stride;
    a.dsum_stride = p->dsum ? p->dsum_stride : 0;
    a.dx_stride = p->dx_stride;
    return cuda_status(launch_rms_norm_backward(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
