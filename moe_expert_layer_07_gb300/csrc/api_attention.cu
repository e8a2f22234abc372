// The C ABI of attention over the four-bit cache and of what goes with it.  As
// in api.cu, everything is checked before anything is enqueued.
#include <math.h>

#include "attention4.cuh"
#include "range.h"

namespace moe {
namespace {

bool al16(const void *p) { return p == nullptr || aligned16(p); }

bool is_float_type(int32_t d) { return d == MOE_OUT_F32 || d == MOE_OUT_BF16; }

bool is_page(int32_t p) { return p == 16 || p == 32 || p == 64 || p == 128; }

int check_cache(const moe_cache4 *c) {
    if (!c || c->pages < 0 || c->kv_heads <= 0 || c->page <= 0 || c->dim <= 0) return MOE_ERR_INVALID_ARG;
    if ((c->dim != 64 && c->dim != 128) || !is_page(c->page) || c->kv_heads > 256 ||
        (int64_t)c->pages * c->page > INT32_MAX)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!al16(c->codes) || !al16(c->scales) || (c->pages > 0 && (!c->codes || !c->scales)))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

int check_attn(const moe_cache_attn *d, const moe_cache4 *cache) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (int rc = check_cache(cache)) return rc;
    if (d->requests < 0 || d->rows < 0 || d->q_heads <= 0 || d->max_pages < 0 || d->max_q < 0 ||
        d->max_len < 0 || d->window < 0 || !isfinite(d->scale))
        return MOE_ERR_INVALID_ARG;
    if (d->requests > kAttnMaxRequests || d->q_heads % cache->kv_heads ||
        (int64_t)d->rows * d->q_heads > INT32_MAX)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_cache_tables(int32_t requests, int32_t page, const int32_t *held, const int32_t *new_tokens,
                     const int32_t *free_pages, int32_t free_count, const int64_t *free_range,
                     int32_t *table, int32_t max_pages, int32_t *lengths, int32_t *starts,
                     int32_t *slots, int32_t *positions, int32_t max_tokens, int64_t *free_out,
                     int32_t *dev_status, void *stream) {
    Range range("moe_cache_tables");
    if (requests < 0 || page <= 0 || free_count < 0 || max_pages < 0 || max_tokens < 0) return MOE_ERR_INVALID_ARG;
    if (!is_page(page) || requests > 16384) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!starts || !free_range || !free_out) return MOE_ERR_INVALID_ARG;
    if (requests > 0 && (!held || !new_tokens || !lengths || (max_pages > 0 && !table))) return MOE_ERR_INVALID_ARG;
    if ((max_tokens > 0 && (!slots || !positions)) || (free_count > 0 && !free_pages)) return MOE_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(held), static_cast<const void *>(new_tokens),
                          static_cast<const void *>(free_pages), static_cast<const void *>(free_range),
                          static_cast<const void *>(table), static_cast<const void *>(lengths),
                          static_cast<const void *>(starts), static_cast<const void *>(slots),
                          static_cast<const void *>(positions), static_cast<const void *>(free_out)})
        if (!al16(p)) return MOE_ERR_INVALID_ARG;
    return launch_cache_tables(requests, page, held, new_tokens, free_pages, free_count, free_range, table,
                               max_pages, lengths, starts, slots, positions, max_tokens, free_out,
                               dev_status, static_cast<cudaStream_t>(stream));
}

int moe_qk_norm_rope(const moe_qk_rope *d, int32_t T, const void *qkv, const int32_t *positions,
                     const float *cos_sin, const void *w_q, const void *w_k, void *q_out, void *k_out,
                     const moe_cache4 *cache, const int32_t *slots, int32_t *dev_status, void *stream) {
    Range range("moe_qk_norm_rope");
    if (!d || T < 0 || d->q_heads <= 0 || d->kv_heads <= 0 || d->dim <= 0 || d->rope_dim < 0)
        return MOE_ERR_INVALID_ARG;
    if (d->style != MOE_ROPE_HALVES && d->style != MOE_ROPE_PAIRS) return MOE_ERR_INVALID_ARG;
    if (!is_float_type(d->param_dtype) || !(d->eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
    if ((d->dim != 64 && d->dim != 128) || d->rope_dim % 16 || d->rope_dim > d->dim ||
        d->q_heads > 65536 || d->kv_heads > 65536 || d->qkv_stride % 8)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (d->qkv_stride < ((int64_t)d->q_heads + 2 * (int64_t)d->kv_heads) * d->dim) return MOE_ERR_INVALID_ARG;
    if (cache) {
        if (int rc = check_cache(cache)) return rc;
        if (cache->dim != d->dim || cache->kv_heads != d->kv_heads) return MOE_ERR_INVALID_ARG;
    }
    if (T == 0) return MOE_OK;
    if (!qkv || !q_out || (!k_out && !cache) || (cache != nullptr) != (slots != nullptr)) return MOE_ERR_INVALID_ARG;
    if (d->rope_dim > 0 && (!positions || !cos_sin || d->max_positions <= 0)) return MOE_ERR_INVALID_ARG;
    for (const void *p : {qkv, static_cast<const void *>(positions), static_cast<const void *>(cos_sin), w_q, w_k,
                          static_cast<const void *>(q_out), static_cast<const void *>(k_out),
                          static_cast<const void *>(slots)})
        if (!al16(p)) return MOE_ERR_INVALID_ARG;
    return launch_qk_norm_rope(d, T, qkv, positions, cos_sin, w_q, w_k, q_out, k_out, cache, slots, dev_status,
                               static_cast<cudaStream_t>(stream));
}

int moe_cache_read(const moe_cache4 *cache, int32_t n, const int32_t *slots, void *k, void *v,
                   int32_t *dev_status, void *stream) {
    Range range("moe_cache_read");
    if (int rc = check_cache(cache)) return rc;
    if (n < 0) return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    if (!slots || (!k && !v) || !al16(slots) || !al16(k) || !al16(v)) return MOE_ERR_INVALID_ARG;
    return launch_cache_read(cache, n, slots, k, v, dev_status, static_cast<cudaStream_t>(stream));
}

int moe_cache_attention_workspace_size(const moe_cache_attn *d, const moe_cache4 *cache, size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    if (int rc = check_attn(d, cache)) return rc;
    *bytes = attention4_workspace(d, cache);
    return MOE_OK;
}

int moe_cache_attention(const moe_cache_attn *d, const moe_cache4 *cache, const void *q, const int32_t *table,
                        const int32_t *lengths, const int32_t *starts, void *out, int32_t out_dtype, float *lse,
                        void *ws, size_t ws_bytes, int32_t *dev_status, void *stream) {
    Range range("moe_cache_attention");
    if (int rc = check_attn(d, cache)) return rc;
    if (!is_float_type(out_dtype)) return MOE_ERR_INVALID_ARG;
    if (d->requests == 0 || d->rows == 0) return MOE_OK;
    if (!q || !lengths || !starts || !out || !ws || (d->max_pages > 0 && !table)) return MOE_ERR_INVALID_ARG;
    if (out == q && out_dtype != MOE_OUT_BF16) return MOE_ERR_INVALID_ARG;
    for (const void *p : {q, static_cast<const void *>(table), static_cast<const void *>(lengths),
                          static_cast<const void *>(starts), static_cast<const void *>(out),
                          static_cast<const void *>(lse), static_cast<const void *>(ws)})
        if (!al16(p)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < attention4_workspace(d, cache)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    return launch_attention4(d, cache, q, table, lengths, starts, out, out_dtype, lse, ws, dev_status,
                             static_cast<cudaStream_t>(stream));
}

int moe_w4_matvec(const moe_w4 *d, int32_t T, const void *x, const void *codes, const void *scales,
                  const void *zeros, void *y, int32_t out_dtype, void *stream) {
    Range range("moe_w4_matvec");
    if (!d || T < 0 || d->n_out <= 0 || d->k_dim <= 0 || !is_float_type(out_dtype)) return MOE_ERR_INVALID_ARG;
    if (d->kind != MOE_W4_MX && d->kind != MOE_W4_INT) return MOE_ERR_INVALID_ARG;
    if (d->kind == MOE_W4_INT ? !is_float_type(d->scale_dtype) : zeros != nullptr) return MOE_ERR_INVALID_ARG;
    if (d->group != 32 && (d->kind == MOE_W4_MX || (d->group != 64 && d->group != 128)))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T > 16 || d->k_dim % d->group || d->k_dim > 32768 || d->n_out > 1 << 30)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!x || !codes || !scales || !y) return MOE_ERR_INVALID_ARG;
    if (!al16(x) || !al16(codes) || !al16(scales) || !al16(zeros) || !al16(y)) return MOE_ERR_INVALID_ARG;
    return launch_w4_matvec(d, T, x, codes, scales, zeros, y, out_dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
