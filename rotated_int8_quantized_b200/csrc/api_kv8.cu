// api_kv8.cu -- the C ABI of the attention-side entry points: argument
// checks on the host and the launches (kernels in kv8.cu and attn_kv8.cu).
// Part of the library's one translation unit, after api.cu.
#include <cmath>

#include "kv8.h"

namespace {

constexpr int32_t kMaxHeads = 4096;
constexpr int64_t kMaxHeadRows = 0x7FFFFFFF;

bool head_dim_ok(int32_t d) { return d == 64 || d == 128; }

convrot_status_t check_kv8(const convrot_kv8_t *c) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return CONVROT_ERR_INVALID_ARG;
    if (c->pages < 1 || c->kv_heads < 1 || c->page_tokens < 1) return CONVROT_ERR_INVALID_ARG;
    if (!head_dim_ok(c->head_dim) || !is_pow2(c->page_tokens) || c->page_tokens < convrot::kKvBlock ||
        c->page_tokens > 1024 || c->kv_heads > kMaxHeads || c->pages > 0x7FFFFFFF ||
        c->pages * c->kv_heads * (c->page_tokens / convrot::kKvBlock) > 0x7FFFFFFF)     // blocks are counted in 32 bits
        return CONVROT_ERR_UNSUPPORTED_SHAPE;
    // keys are read 32 bytes at a time
    if (((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 31u) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
        return CONVROT_ERR_ALIGNMENT;
    return CONVROT_OK;
}

// Rows of heads a kernel reads: any strides that keep 16-byte rows.
convrot_status_t check_rows(const void *p, int64_t ts, int64_t hs) {
    if (!p || ts < 0 || hs < 0) return CONVROT_ERR_INVALID_ARG;
    if (!aligned16(p) || ts % 8 != 0 || hs % 8 != 0) return CONVROT_ERR_ALIGNMENT;
    return CONVROT_OK;
}

// Rows a kernel writes: two of them never overlap.
convrot_status_t check_rows_out(const void *p, int64_t ts, int64_t hs, int64_t tokens, int64_t heads, int64_t dim) {
    const convrot_status_t s = check_rows(p, ts, hs);
    if (s != CONVROT_OK) return s;
    const bool heads_inside = (heads == 1 || hs >= dim) && (tokens == 1 || ts >= (heads - 1) * hs + dim);
    const bool tokens_inside = (tokens == 1 || ts >= dim) && (heads == 1 || hs >= (tokens - 1) * ts + dim);
    return heads_inside || tokens_inside ? CONVROT_OK : CONVROT_ERR_INVALID_ARG;
}

convrot_status_t check_rope(const convrot_rope_t *r, const int32_t *positions, int32_t dim, bool needs_positions,
                            convrot::RopeArgs *out) {
    *out = convrot::RopeArgs{};
    if (!r) return CONVROT_OK;
    if (!r->cos_sin || r->positions < 1 || r->axes < 1 || r->axes > 8) return CONVROT_ERR_INVALID_ARG;
    if (needs_positions && !positions) return CONVROT_ERR_INVALID_ARG;
    if (!positions && (r->axis || r->axes != 1)) return CONVROT_ERR_INVALID_ARG;
    if (r->rot_dim < 8 || r->rot_dim > dim || r->rot_dim % 8 != 0) return CONVROT_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(r->cos_sin) || ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(r->axis)) & 3u))
        return CONVROT_ERR_ALIGNMENT;
    out->cs = r->cos_sin;
    out->rows = r->positions;
    out->axis = r->axis;
    out->pos = positions;
    out->rot = r->rot_dim;
    out->adjacent = r->adjacent != 0;
    out->axes = r->axes;
    return CONVROT_OK;
}

convrot_status_t check_norm(const void *qw, const void *kw, float eps) {
    if ((qw && !aligned16(qw)) || (kw && !aligned16(kw))) return CONVROT_ERR_ALIGNMENT;
    return eps >= 0.f && std::isfinite(eps) ? CONVROT_OK : CONVROT_ERR_INVALID_ARG;
}

convrot_status_t check_seqs(const convrot_kv8_seqs_t *s, const convrot_kv8_t *c, int64_t heads, convrot::KvSeqs *out) {
    if (!s->page_table || !s->kv_len || s->batch < 1 || s->max_pages < 1 || s->tokens < 1) return CONVROT_ERR_INVALID_ARG;
    if (!s->cu && s->tokens != s->batch) return CONVROT_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(s->page_table) | reinterpret_cast<uintptr_t>(s->kv_len) |
         reinterpret_cast<uintptr_t>(s->cu)) & 3u)
        return CONVROT_ERR_ALIGNMENT;
    // grids: one CTA for a block of a head at the most
    if (s->tokens > kMaxHeadRows || s->tokens * heads > kMaxHeadRows || ((int64_t)s->tokens / 16 + 2 * (int64_t)s->batch) * heads > kMaxHeadRows / 2)
        return CONVROT_ERR_UNSUPPORTED_SHAPE;
    out->table = s->page_table;
    out->kv_len = s->kv_len;
    out->cu = s->cu;
    out->tokens = s->tokens;
    out->pages = c->pages;
    out->batch = s->batch;
    out->max_pages = s->max_pages;
    out->page_shift = 0;
    while ((1 << out->page_shift) < c->page_tokens) ++out->page_shift;
    return CONVROT_OK;
}

convrot::KvCache cache_args(const convrot_kv8_t *c) {
    return {c->k, c->v, c->k_scale, c->v_scale, c->kv_heads, c->head_dim};
}

convrot::HeadRows rows_in(const void *p, int64_t ts, int64_t hs) { return {static_cast<const uint16_t *>(p), ts, hs}; }
convrot::HeadRowsOut rows_out(void *p, int64_t ts, int64_t hs) { return {static_cast<uint16_t *>(p), ts, hs}; }

convrot_status_t check_attn(const convrot_attn_kv8_t *job, convrot::AttnArgs *a) {
    if (!job) return CONVROT_ERR_INVALID_ARG;
    convrot_status_t s = check_kv8(job->cache);
    if (s != CONVROT_OK) return s;
    if (job->q_heads < 1 || !job->out || !(job->scale > 0.f) || !std::isfinite(job->scale)) return CONVROT_ERR_INVALID_ARG;
    if (job->q_heads > kMaxHeads || job->q_heads % job->cache->kv_heads != 0) return CONVROT_ERR_UNSUPPORTED_SHAPE;
    if ((s = check_rows(job->q, job->q_token_stride, job->q_head_stride)) != CONVROT_OK) return s;
    if (!aligned16(job->out) || (reinterpret_cast<uintptr_t>(job->lse) & 3u)) return CONVROT_ERR_ALIGNMENT;
    if ((s = check_seqs(&job->seqs, job->cache, job->q_heads, &a->s)) != CONVROT_OK) return s;
    a->c = cache_args(job->cache);
    a->q_heads = job->q_heads;
    a->q = rows_in(job->q, job->q_token_stride, job->q_head_stride);
    a->out = static_cast<uint16_t *>(job->out);
    a->lse = job->lse;
    a->scale = job->scale;
    a->causal = job->causal != 0;
    a->ws = nullptr;
    return CONVROT_OK;
}

size_t attn_bytes(const convrot::AttnArgs &a, int sms) {
    return round256((size_t)convrot::attn_kv8_workspace_bytes(a, sms));
}

}  // namespace

#pragma GCC visibility push(default)
extern "C" {

convrot_status_t convrot_kv8_init(convrot_kv8_t *c, int8_t *k, int8_t *v, float *k_scale, float *v_scale, int64_t pages,
                                  int32_t kv_heads, int32_t page_tokens, int32_t head_dim) {
    if (!c) return CONVROT_ERR_INVALID_ARG;
    const convrot_kv8_t t = {k, v, k_scale, v_scale, pages, kv_heads, page_tokens, head_dim};
    const convrot_status_t s = check_kv8(&t);
    if (s == CONVROT_OK) *c = t;
    return s;
}

convrot_status_t convrot_qk_norm_rope(const convrot_qk_norm_rope_t *j, void *stream) {
    if (!j || j->tokens < 1 || j->q_heads < 1 || j->kv_heads < 0) return CONVROT_ERR_INVALID_ARG;
    if (!head_dim_ok(j->head_dim) || j->q_heads > kMaxHeads || j->kv_heads > kMaxHeads ||
        j->tokens > kMaxHeadRows / (j->q_heads + j->kv_heads))
        return CONVROT_ERR_UNSUPPORTED_SHAPE;
    convrot::NormRopeArgs a = {};
    convrot_status_t s;
    if ((s = check_rows(j->q, j->q_token_stride, j->q_head_stride)) != CONVROT_OK) return s;
    if ((s = check_rows_out(j->q_out, j->q_out_token_stride, j->q_out_head_stride, j->tokens, j->q_heads, j->head_dim)) !=
        CONVROT_OK)
        return s;
    if (j->kv_heads) {
        if ((s = check_rows(j->k, j->k_token_stride, j->k_head_stride)) != CONVROT_OK) return s;
        if ((s = check_rows_out(j->k_out, j->k_out_token_stride, j->k_out_head_stride, j->tokens, j->kv_heads,
                                j->head_dim)) != CONVROT_OK)
            return s;
    }
    if ((s = check_norm(j->q_weight, j->k_weight, j->eps)) != CONVROT_OK) return s;
    if ((s = check_rope(j->rope, j->positions, j->head_dim, true, &a.rope)) != CONVROT_OK) return s;
    a.tokens = j->tokens;
    a.q_heads = j->q_heads;
    a.kv_heads = j->kv_heads;
    a.dim = j->head_dim;
    a.q = rows_in(j->q, j->q_token_stride, j->q_head_stride);
    a.k = rows_in(j->k, j->k_token_stride, j->k_head_stride);
    a.q_out = rows_out(j->q_out, j->q_out_token_stride, j->q_out_head_stride);
    a.k_out = rows_out(j->k_out, j->k_out_token_stride, j->k_out_head_stride);
    a.qw = static_cast<const uint16_t *>(j->q_weight);
    a.kw = static_cast<const uint16_t *>(j->k_weight);
    a.eps = j->eps;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != CONVROT_OK) return s;
    return from_cuda(convrot::launch_norm_rope(a, dev.num_sms, static_cast<cudaStream_t>(stream)));
}

convrot_status_t convrot_kv8_append(const convrot_kv8_append_t *j, void *stream) {
    if (!j) return CONVROT_ERR_INVALID_ARG;
    convrot_status_t s = check_kv8(j->cache);
    if (s != CONVROT_OK) return s;
    if (j->q_heads < 0) return CONVROT_ERR_INVALID_ARG;
    if (j->q_heads > kMaxHeads) return CONVROT_ERR_UNSUPPORTED_SHAPE;
    const int32_t dim = j->cache->head_dim;
    convrot::AppendArgs a = {};
    if ((s = check_seqs(&j->seqs, j->cache, (int64_t)j->q_heads + j->cache->kv_heads, &a.s)) != CONVROT_OK) return s;
    if ((s = check_rows(j->k, j->k_token_stride, j->k_head_stride)) != CONVROT_OK) return s;
    if ((s = check_rows(j->v, j->v_token_stride, j->v_head_stride)) != CONVROT_OK) return s;
    if (j->q_heads) {
        if ((s = check_rows(j->q, j->q_token_stride, j->q_head_stride)) != CONVROT_OK) return s;
        if ((s = check_rows_out(j->q_out, j->q_out_token_stride, j->q_out_head_stride, j->seqs.tokens, j->q_heads, dim)) !=
            CONVROT_OK)
            return s;
    }
    if ((s = check_norm(j->q_weight, j->k_weight, j->eps)) != CONVROT_OK) return s;
    if ((s = check_rope(j->rope, j->positions, dim, false, &a.rope)) != CONVROT_OK) return s;
    a.c = cache_args(j->cache);
    a.q_heads = j->q_heads;
    a.q = rows_in(j->q, j->q_token_stride, j->q_head_stride);
    a.k = rows_in(j->k, j->k_token_stride, j->k_head_stride);
    a.v = rows_in(j->v, j->v_token_stride, j->v_head_stride);
    a.q_out = rows_out(j->q_out, j->q_out_token_stride, j->q_out_head_stride);
    a.qw = static_cast<const uint16_t *>(j->q_weight);
    a.kw = static_cast<const uint16_t *>(j->k_weight);
    a.eps = j->eps;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != CONVROT_OK) return s;
    return from_cuda(convrot::launch_kv8_append(a, dev.num_sms, static_cast<cudaStream_t>(stream)));
}

convrot_status_t convrot_kv8_read(const convrot_kv8_read_t *j, void *stream) {
    if (!j) return CONVROT_ERR_INVALID_ARG;
    convrot_status_t s = check_kv8(j->cache);
    if (s != CONVROT_OK) return s;
    if (!j->k_out && !j->v_out) return CONVROT_ERR_INVALID_ARG;
    convrot::ReadArgs a = {};
    if ((s = check_seqs(&j->seqs, j->cache, j->cache->kv_heads, &a.s)) != CONVROT_OK) return s;
    if (!aligned16(j->k_out) || !aligned16(j->v_out)) return CONVROT_ERR_ALIGNMENT;
    a.c = cache_args(j->cache);
    a.k_out = static_cast<uint16_t *>(j->k_out);
    a.v_out = static_cast<uint16_t *>(j->v_out);
    DeviceInfo dev;
    if ((s = current_device(&dev)) != CONVROT_OK) return s;
    return from_cuda(convrot::launch_kv8_read(a, dev.num_sms, static_cast<cudaStream_t>(stream)));
}

size_t convrot_attn_kv8_workspace_bytes(const convrot_attn_kv8_t *job) {
    convrot::AttnArgs a = {};
    return check_attn(job, &a) == CONVROT_OK ? attn_bytes(a, sms_for_sizing()) : 0;
}

convrot_status_t convrot_attn_kv8(const convrot_attn_kv8_t *job, void *ws, size_t ws_bytes, void *stream) {
    convrot::AttnArgs a = {};
    convrot_status_t s = check_attn(job, &a);
    if (s != CONVROT_OK) return s;
    if (ws && !aligned16(ws)) return CONVROT_ERR_ALIGNMENT;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != CONVROT_OK) return s;
    if (!ws || ws_bytes < attn_bytes(a, dev.num_sms)) return CONVROT_ERR_WORKSPACE;
    a.ws = ws;
    return from_cuda(convrot::launch_attn_kv8(a, dev.num_sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
#pragma GCC visibility pop
