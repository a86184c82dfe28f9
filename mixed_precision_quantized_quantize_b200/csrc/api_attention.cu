// api_attention.cu -- the extern "C" entry points of the attention between a
// layer's QKV and output projections (include/quik.h): argument validation
// and dispatch.  No device memory is allocated here.
#include <cmath>
#include <cstdint>

#include "quik_internal.h"

namespace {

constexpr int kMaxHeads = 4096;
constexpr int kMaxSequences = 65535;  // a grid dimension

inline bool aligned(const void *p, unsigned to) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}
inline bool ok_dim(int d) { return d == 64 || d == 128; }
// rows of `heads` heads: 16-byte units
inline bool ok_rows(const void *p, int64_t stride, int64_t heads, int64_t dim) {
    return aligned(p, 16) && stride % 8 == 0 && stride >= heads * dim;
}

quik_status check_heads(const quik_heads *s) {
    if (s == nullptr || s->tokens < 0 || s->q_heads < 0 || s->kv_heads < 0) return QUIK_ERR_INVALID_ARG;
    if (s->interleaved != 0 && s->interleaved != 1) return QUIK_ERR_INVALID_ARG;
    if (s->rotary_dim < 0 || s->rotary_dim % 16 != 0) return QUIK_ERR_INVALID_ARG;
    if (s->rotary_dim > 0 && s->table_rows < 1) return QUIK_ERR_INVALID_ARG;
    if (!ok_dim(s->head_dim)) return s->head_dim < 1 ? QUIK_ERR_INVALID_ARG : QUIK_ERR_UNSUPPORTED;
    if (s->rotary_dim > s->head_dim) return QUIK_ERR_INVALID_ARG;
    if (s->q_heads > kMaxHeads || s->kv_heads > kMaxHeads) return QUIK_ERR_UNSUPPORTED;
    return QUIK_OK;
}

quik_status check_rotation(const quik_heads *s, const float *cos, const float *sin,
                           const int32_t *positions, quik::RotaryArgs *out) {
    out->rotary = s->rotary_dim;
    out->rows = s->table_rows;
    out->interleaved = s->interleaved != 0;
    if (s->rotary_dim == 0) return QUIK_OK;
    if (!aligned(cos, 16) || !aligned(sin, 16) || !aligned(positions, 4)) return QUIK_ERR_INVALID_ARG;
    out->cos = cos;
    out->sin = sin;
    out->positions = positions;
    return QUIK_OK;
}

quik_status check_cache(const quik_kv_cache *c) {
    if (c == nullptr || c->heads < 1 || c->pages < 1 || c->reserved != 0) return QUIK_ERR_INVALID_ARG;
    if (c->kv_type < QUIK_KV_FP16 || c->kv_type > QUIK_KV_INT4) return QUIK_ERR_INVALID_ARG;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
        return QUIK_ERR_INVALID_ARG;
    if (!ok_dim(c->head_dim)) return c->head_dim < 1 ? QUIK_ERR_INVALID_ARG : QUIK_ERR_UNSUPPORTED;
    if (c->heads > kMaxHeads) return QUIK_ERR_UNSUPPORTED;
    return QUIK_OK;
}

bool ok_buffers(const quik_kv_cache *c) {
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return false;
    return c->kv_type == QUIK_KV_FP16 || (aligned(c->k_scale, 16) && aligned(c->v_scale, 16));
}

quik_status check_attention(const quik_attention *a, const quik_kv_cache *cache) {
    quik_status st = check_cache(cache);
    if (st != QUIK_OK) return st;
    if (a == nullptr || a->tokens < 0 || a->sequences < 0 || a->max_tokens < 0 || a->max_context < 0 ||
        a->max_pages < 0 || a->mask_words < 0 || !std::isfinite(a->scale))
        return QUIK_ERR_INVALID_ARG;
    if (a->q_heads < 1 || a->q_heads % cache->heads != 0) return QUIK_ERR_INVALID_ARG;
    if (a->q_heads > kMaxHeads || a->sequences > kMaxSequences) return QUIK_ERR_UNSUPPORTED;
    return QUIK_OK;
}

inline bool no_work(const quik_attention *a) {
    return a->tokens == 0 || a->sequences == 0 || a->max_tokens == 0;
}

quik::AttentionArgs args_of(const quik_attention *a, const quik_kv_cache *cache) {
    quik::AttentionArgs r{};
    r.tokens = a->tokens;
    r.sequences = a->sequences;
    r.q_heads = a->q_heads;
    // no sequence has more new tokens than there are rows
    r.max_tokens = a->max_tokens < a->tokens ? a->max_tokens : a->tokens;
    r.max_pages = a->max_pages;
    r.max_context = a->max_context;
    r.mask_words = a->mask_words;
    r.scale = a->scale;
    r.cache = *cache;
    return r;
}

}  // namespace

extern "C" {

quik_status quik_qk_norm_rope(const quik_heads *heads, const void *q, int64_t q_stride, const void *k,
                              int64_t k_stride, const void *q_gamma, const void *k_gamma, float eps,
                              const float *cos_table, const float *sin_table,
                              const int32_t *positions, void *q_out, int64_t q_out_stride,
                              void *k_out, int64_t k_out_stride, quik_stream_t stream) {
    quik_status st = check_heads(heads);
    if (st != QUIK_OK) return st;
    if (heads->q_heads + heads->kv_heads == 0) return QUIK_ERR_INVALID_ARG;
    // nothing of a side without heads is used (the kernel takes the lanes past the
    // last row for rows of k, and would read its weight)
    if (heads->q_heads == 0) q_gamma = nullptr;
    if (heads->kv_heads == 0) k_gamma = nullptr;
    if ((q_gamma != nullptr || k_gamma != nullptr) && !(std::isfinite(eps) && eps > 0.0f))
        return QUIK_ERR_INVALID_ARG;
    if ((q_gamma != nullptr && !aligned(q_gamma, 16)) || (k_gamma != nullptr && !aligned(k_gamma, 16)))
        return QUIK_ERR_INVALID_ARG;
    if (heads->tokens == 0) return QUIK_OK;
    quik::QkArgs a{};
    if ((st = check_rotation(heads, cos_table, sin_table, positions, &a.rot)) != QUIK_OK) return st;
    const int d = heads->head_dim;
    if (heads->q_heads > 0 && (!ok_rows(q, q_stride, heads->q_heads, d) ||
                               !ok_rows(q_out, q_out_stride, heads->q_heads, d)))
        return QUIK_ERR_INVALID_ARG;
    if (heads->kv_heads > 0 && (!ok_rows(k, k_stride, heads->kv_heads, d) ||
                                !ok_rows(k_out, k_out_stride, heads->kv_heads, d)))
        return QUIK_ERR_INVALID_ARG;
    // in place only row by row
    if ((heads->q_heads > 0 && q == q_out && q_stride != q_out_stride) ||
        (heads->kv_heads > 0 && k == k_out && k_stride != k_out_stride))
        return QUIK_ERR_INVALID_ARG;
    a.tokens = heads->tokens;
    a.q_heads = heads->q_heads;
    a.kv_heads = heads->kv_heads;
    a.head_dim = d;
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_gamma = static_cast<const uint16_t *>(q_gamma);
    a.k_gamma = static_cast<const uint16_t *>(k_gamma);
    a.eps = eps;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.k_out = static_cast<uint16_t *>(k_out);
    a.q_out_stride = q_out_stride;
    a.k_out_stride = k_out_stride;
    return quik::launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? QUIK_OK
                                                                                        : QUIK_ERR_CUDA;
}

quik_status quik_kv_append(const quik_heads *heads, const quik_kv_cache *cache, const void *k,
                           int64_t k_stride, const void *v, int64_t v_stride, const float *cos_table,
                           const float *sin_table, const int32_t *positions, const int64_t *slots,
                           quik_stream_t stream) {
    quik_status st = check_heads(heads);
    if (st != QUIK_OK) return st;
    if ((st = check_cache(cache)) != QUIK_OK) return st;
    if (heads->kv_heads != cache->heads || heads->head_dim != cache->head_dim) return QUIK_ERR_INVALID_ARG;
    if (!ok_buffers(cache)) return QUIK_ERR_INVALID_ARG;
    if (heads->tokens == 0) return QUIK_OK;
    quik::AppendArgs a{};
    if ((st = check_rotation(heads, cos_table, sin_table, positions, &a.rot)) != QUIK_OK) return st;
    if (!ok_rows(k, k_stride, cache->heads, cache->head_dim) ||
        !ok_rows(v, v_stride, cache->heads, cache->head_dim) || !aligned(slots, 8))
        return QUIK_ERR_INVALID_ARG;
    a.tokens = heads->tokens;
    a.cache = *cache;
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slots = slots;
    return quik::launch_kv_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? QUIK_OK
                                                                                     : QUIK_ERR_CUDA;
}

quik_status quik_kv_gather(const quik_kv_cache *cache, int32_t tokens, const int64_t *slots, void *k_out,
                           int64_t k_stride, void *v_out, int64_t v_stride, quik_stream_t stream) {
    quik_status st = check_cache(cache);
    if (st != QUIK_OK) return st;
    if (tokens < 0 || !ok_buffers(cache)) return QUIK_ERR_INVALID_ARG;
    if (tokens == 0) return QUIK_OK;
    if (!ok_rows(k_out, k_stride, cache->heads, cache->head_dim) ||
        !ok_rows(v_out, v_stride, cache->heads, cache->head_dim) || !aligned(slots, 8))
        return QUIK_ERR_INVALID_ARG;
    quik::GatherArgs a{};
    a.tokens = tokens;
    a.cache = *cache;
    a.slots = slots;
    a.k_out = static_cast<uint16_t *>(k_out);
    a.v_out = static_cast<uint16_t *>(v_out);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    return quik::launch_kv_gather(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? QUIK_OK
                                                                                     : QUIK_ERR_CUDA;
}

size_t quik_attention_workspace_size(const quik_attention *attention, const quik_kv_cache *cache) {
    if (check_attention(attention, cache) != QUIK_OK || no_work(attention)) return 0;
    return quik::attention_workspace(args_of(attention, cache));
}

quik_status quik_tree_attention(const quik_attention *attention, const quik_kv_cache *cache,
                                const void *q, int64_t q_stride, const int32_t *page_table,
                                const int32_t *context, const int32_t *cu_tokens,
                                const uint32_t *tree_mask, void *out, int64_t out_stride, float *lse,
                                void *workspace, size_t workspace_bytes, quik_stream_t stream) {
    quik_status st = check_attention(attention, cache);
    if (st != QUIK_OK) return st;
    if (!ok_buffers(cache)) return QUIK_ERR_INVALID_ARG;
    if (no_work(attention)) return QUIK_OK;
    quik::AttentionArgs a = args_of(attention, cache);
    if (!ok_rows(q, q_stride, a.q_heads, cache->head_dim) ||
        !ok_rows(out, out_stride, a.q_heads, cache->head_dim))
        return QUIK_ERR_INVALID_ARG;
    if (!aligned(context, 4) || !aligned(cu_tokens, 4) || (lse != nullptr && !aligned(lse, 4)))
        return QUIK_ERR_INVALID_ARG;
    if (a.max_pages > 0 && !aligned(page_table, 4)) return QUIK_ERR_INVALID_ARG;
    if (tree_mask != nullptr &&
        (!aligned(tree_mask, 4) || static_cast<int64_t>(a.mask_words) * 32 < a.max_tokens))
        return QUIK_ERR_INVALID_ARG;
    const size_t need = quik::attention_workspace(a);
    if (need > 0 && (!aligned(workspace, 16) || workspace_bytes < need)) return QUIK_ERR_INVALID_ARG;
    a.q = static_cast<const uint16_t *>(q);
    a.q_stride = q_stride;
    a.page_table = page_table;
    a.context = context;
    a.cu_tokens = cu_tokens;
    a.mask = tree_mask;
    a.out = static_cast<uint16_t *>(out);
    a.out_stride = out_stride;
    a.lse = lse;
    a.partial = static_cast<float *>(workspace);
    return quik::launch_tree_attention(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
