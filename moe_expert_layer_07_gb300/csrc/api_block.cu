// The C ABI of what stands around the layer: the few-token layer, MXFP4 and
// the norms around a block.  As in api.cu, everything is checked before
// anything is enqueued.
#include "internal.h"
#include "range.h"

namespace moe {
namespace {

bool al16(const void *p) { return p == nullptr || aligned16(p); }

// products write 32 bytes at a time
bool al32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

bool is_float_type(int32_t d) { return d == MOE_OUT_F32 || d == MOE_OUT_BF16; }

// check_config, with MXFP4 as a third dtype (its shape rules are BF16's) and
// the few-token bound.
int check_few(const moe_config *cfg) {
    if (!cfg) return MOE_ERR_INVALID_ARG;
    moe_config c = *cfg;
    if (c.dtype == MOE_DTYPE_MXFP4) c.dtype = MOE_DTYPE_BF16;
    if (int rc = check_config(&c)) return rc;
    return c.max_tokens > kFewMaxTokens ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}

int check_mx4_gemm(int32_t groups, int32_t n_out, int32_t k_dim, int32_t rows) {
    if (groups <= 0 || n_out <= 0 || k_dim <= 0 || rows < 0) return MOE_ERR_INVALID_ARG;
    if (groups > 1024 || n_out % 128 || k_dim % 128) return MOE_ERR_UNSUPPORTED_SHAPE;
    // tiles, and a CTA's steps of 256 along K, are counted in 32 bits
    const int64_t tiles = ((int64_t)n_out + 255) / 256 * (groups + (int64_t)rows / 128 + 1);
    if (tiles > INT32_MAX || tiles * ((k_dim + 255) / 256) > INT32_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uint8_t *p = static_cast<const uint8_t *>(a), *q = static_cast<const uint8_t *>(b);
    return p && q && p < q + nb && q < p + na;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int32_t moe_layer_few_max_tokens(void) { return kFewMaxTokens; }

int moe_layer_few_layout(const moe_config *cfg, moe_few_layout *L) {
    if (int rc = check_few(cfg)) return rc;
    if (!L) return MOE_ERR_INVALID_ARG;
    few_layout(cfg, L);
    return MOE_OK;
}

int moe_layer_few_workspace_size(const moe_config *cfg, size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    moe_few_layout L;
    if (int rc = moe_layer_few_layout(cfg, &L)) return rc;
    *bytes = L.total;
    return MOE_OK;
}

int moe_layer_few(const moe_config *cfg, const moe_weights *w, int32_t T, const void *x, void *out,
                  int32_t out_dtype, void *ws, size_t ws_bytes, void *stream) {
    Range range("moe_layer_few");
    if (int rc = check_few(cfg)) return rc;
    if (!w || !ws || T < 0 || T > cfg->max_tokens || !is_float_type(out_dtype))
        return MOE_ERR_INVALID_ARG;
    const bool scaled = cfg->dtype != MOE_DTYPE_BF16;
    if (T > 0 && (!x || !out)) return MOE_ERR_INVALID_ARG;
    if (!w->w_gate || !w->w13 || !w->w2 || (scaled && (!w->w13_scales || !w->w2_scales)))
        return MOE_ERR_INVALID_ARG;
    if (w->e_bias && cfg->scoring != MOE_SCORING_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (w->expert_layout != MOE_LAYOUT_TILES) return MOE_ERR_INVALID_ARG;
    if (!al16(x) || !al16(out) || !al16(ws) || !al16(w->w_gate) || !al16(w->w13) || !al16(w->w2))
        return MOE_ERR_INVALID_ARG;
    if (cfg->dtype == MOE_DTYPE_MXFP4 && (!al16(w->w13_scales) || !al16(w->w2_scales)))
        return MOE_ERR_INVALID_ARG;
    moe_few_layout L;
    few_layout(cfg, &L);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        MOE_CUDA_TRY(cudaMemsetAsync(ws, 0, 4, s));   // the status word
        return MOE_OK;
    }
    return launch_layer_few(cfg, w, T, x, out, out_dtype, ws, s);
}

int moe_mx4_quantize(int32_t rows, int32_t cols, const void *in, int32_t in_dtype, void *codes,
                     void *scales, void *stream) {
    Range range("moe_mx4_quantize");
    if (rows < 0 || cols <= 0 || !is_float_type(in_dtype)) return MOE_ERR_INVALID_ARG;
    if (cols % 32) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!in || !codes || !scales || !al16(in) || !al16(codes)) return MOE_ERR_INVALID_ARG;
    return launch_mx4_quantize(rows, cols, in, in_dtype == MOE_OUT_F32, codes, scales,
                               static_cast<cudaStream_t>(stream));
}

int moe_mx4_dequantize(int32_t rows, int32_t cols, const void *codes, const void *scales, void *out,
                       int32_t out_dtype, void *stream) {
    Range range("moe_mx4_dequantize");
    if (rows < 0 || cols <= 0 || !is_float_type(out_dtype)) return MOE_ERR_INVALID_ARG;
    if (cols % 32) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!codes || !scales || !out || !al16(codes) || !al16(out)) return MOE_ERR_INVALID_ARG;
    return launch_mx4_dequantize(rows, cols, codes, scales, out, out_dtype == MOE_OUT_F32,
                                 static_cast<cudaStream_t>(stream));
}

int moe_mx4_pack_weights(int32_t groups, int32_t n_out, int32_t k_dim, const void *codes,
                         const void *scales, void *codes_tiled, void *scales_tiled, void *stream) {
    Range range("moe_mx4_pack_weights");
    if (groups < 0 || n_out <= 0 || k_dim <= 0) return MOE_ERR_INVALID_ARG;
    if (n_out % 128 || k_dim % 128) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (groups == 0) return MOE_OK;
    if (!codes || !scales || !codes_tiled || !scales_tiled) return MOE_ERR_INVALID_ARG;
    if (!al16(codes) || !al16(scales) || !al16(codes_tiled) || !al16(scales_tiled))
        return MOE_ERR_INVALID_ARG;
    const size_t n = (size_t)groups * n_out * k_dim;
    if (overlap(codes, n / 2, codes_tiled, n / 2) || overlap(scales, n / 32, scales_tiled, n / 32))
        return MOE_ERR_INVALID_ARG;
    return launch_mx4_pack(groups, n_out, k_dim, codes, scales, codes_tiled, scales_tiled,
                           static_cast<cudaStream_t>(stream));
}

int moe_mx4_grouped_gemm(int32_t groups, int32_t n_out, int32_t k_dim, int32_t rows, const void *a,
                         const void *a_scales, const int32_t *expert_offsets, const void *w_tiled,
                         const void *w_scales_tiled, void *c, int32_t c_dtype, int32_t *dev_status,
                         void *stream) {
    Range range("moe_mx4_grouped_gemm");
    if (!is_float_type(c_dtype)) return MOE_ERR_INVALID_ARG;
    if (int rc = check_mx4_gemm(groups, n_out, k_dim, rows)) return rc;
    if (rows == 0) return MOE_OK;
    if (!a || !a_scales || !expert_offsets || !w_tiled || !w_scales_tiled || !c)
        return MOE_ERR_INVALID_ARG;
    if (!al16(a) || !al16(a_scales) || !al16(w_tiled) || !al16(w_scales_tiled) || !al32(c))
        return MOE_ERR_INVALID_ARG;
    return launch_mx4_gemm(groups, n_out, k_dim, rows, a, a_scales, expert_offsets, w_tiled,
                           w_scales_tiled, c, c_dtype, dev_status, static_cast<cudaStream_t>(stream));
}

int moe_mx4_grouped_gemm_swiglu(int32_t groups, int32_t inter, int32_t k_dim, int32_t rows,
                                const void *a, const void *a_scales, const int32_t *expert_offsets,
                                const void *w13_tiled, const void *w13_scales_tiled, void *h,
                                void *h_scales, int32_t *dev_status, void *stream) {
    Range range("moe_mx4_grouped_gemm_swiglu");
    if (inter <= 0 || inter > INT32_MAX / 2) return MOE_ERR_INVALID_ARG;
    if (int rc = check_mx4_gemm(groups, 2 * inter, k_dim, rows)) return rc;
    if (inter % 128) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!a || !a_scales || !expert_offsets || !w13_tiled || !w13_scales_tiled || !h || !h_scales)
        return MOE_ERR_INVALID_ARG;
    if (!al16(a) || !al16(a_scales) || !al16(w13_tiled) || !al16(w13_scales_tiled) || !al32(h) ||
        !al16(h_scales))
        return MOE_ERR_INVALID_ARG;
    return launch_mx4_gemm_swiglu(groups, inter, k_dim, rows, a, a_scales, expert_offsets, w13_tiled,
                                  w13_scales_tiled, h, h_scales, dev_status,
                                  static_cast<cudaStream_t>(stream));
}

int moe_block_norm(const moe_norm *d, int32_t T, const void *y, const void *residual,
                   const void *gate, const void *w_post, const void *b_post, const void *w_pre,
                   const void *b_pre, void *residual_out, void *x_out, void *stream) {
    Range range("moe_block_norm");
    if (!d || T < 0 || d->hidden <= 0) return MOE_ERR_INVALID_ARG;
    if (d->kind != MOE_NORM_RMS && d->kind != MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
    if (!is_float_type(d->y_dtype) || !is_float_type(d->residual_dtype) ||
        !is_float_type(d->param_dtype))
        return MOE_ERR_INVALID_ARG;
    if (d->gate_mode < MOE_GATE_NONE || d->gate_mode > MOE_GATE_FULL ||
        (d->gate_mode != MOE_GATE_NONE) != (gate != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (!(d->eps >= 0.0f)) return MOE_ERR_INVALID_ARG;   // NaN too
    if (d->hidden % 8 || d->hidden > 16384) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!y && (gate || w_post)) return MOE_ERR_INVALID_ARG;
    if ((b_post && !w_post) || (b_pre && !w_pre) || (w_pre != nullptr) != (x_out != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!residual || (!residual_out && !x_out)) return MOE_ERR_INVALID_ARG;
    for (const void *p : {y, residual, gate, w_post, b_post, w_pre, b_pre,
                          static_cast<const void *>(residual_out), static_cast<const void *>(x_out)})
        if (!al16(p)) return MOE_ERR_INVALID_ARG;
    return launch_block_norm(d, T, y, residual, gate, w_post, b_post, w_pre, b_pre, residual_out,
                             x_out, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
