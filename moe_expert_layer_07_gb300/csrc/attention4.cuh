// What the attention kernels over the four-bit cache share: the work list of a
// call, and where the results of a piece of a request are kept.
#pragma once

#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"

namespace moe {

constexpr int kAttnMaxRequests = 4096;
constexpr int kAttnTile = 16;      // tokens of a tile
constexpr int kAttnWarps = 8;
constexpr int kAttnChunk = kAttnTile * kAttnWarps;   // tokens of a unit of work

struct AttnArgs {
    const uint16_t *q;
    const uint8_t *codes, *scales;
    const int32_t *table, *lengths, *starts;
    void *out;
    float *lse;
    int32_t *status;
    // partial results, two to a CTA: weighted sums [rows, D], then top and sum of each row
    float *part;
    int32_t *plan;   // [requests + 1]: first unit of each request, then units a CTA
    int B, rows, Hq, Hk, G, max_pages, pages, page_shift, window, out_bf16, ctas;
    int few_rows;    // requests of more rows are another kernel's
    float scale_log2;
};

// Request b of the call: its query rows and the tokens that they see.
struct AttnRequest {
    int row0, n, len;      // n = 0 where there is nothing to compute
    int lo;                // first token seen by any row, a multiple of the tile
    bool bad;
};

__device__ __forceinline__ AttnRequest attn_request(const AttnArgs &a, int b) {
    AttnRequest r;
    r.row0 = a.starts[b];
    const int end = a.starts[b + 1];
    r.len = a.lengths[b];
    r.bad = r.row0 < 0 || end < r.row0 || end > a.rows || r.len < 0 ||
            r.len > (int64_t)a.max_pages << a.page_shift || r.len > INT32_MAX - 1024;
    r.n = r.bad ? 0 : end - r.row0;
    const int first = r.len - r.n;   // position of the first row; may be negative
    r.lo = a.window && first >= a.window ? (first - a.window + 1) / kAttnTile * kAttnTile : 0;
    return r;
}

// Units of work over the request's tokens, for one KV head and group of rows.
__device__ __forceinline__ int attn_chunks(const AttnRequest &r) {
    return max(1, (r.len - r.lo + kAttnChunk - 1) / kAttnChunk);
}

// One row of one head (output row i) from the partial results of CTAs k0 .. k1, in
// order, by a warp; `rows_at_once` rows in each, this the rr-th.
template <int D>
__device__ __forceinline__ void attn_join(const AttnArgs &a, int rows_at_once, int rr, int64_t i, int k0, int k1,
                                          int lane) {
    const int64_t size = (int64_t)rows_at_once * (D + 2);
    float m = -INFINITY;
    for (int k = k0 + lane; k <= k1; k += 32)
        m = fmaxf(m, a.part[(2 * k + (k == k0)) * size + rows_at_once * D + rr]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.0f;
    float v[D / 32];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) v[j] = 0.0f;
#pragma unroll 4
    for (int k = k0; k <= k1; ++k) {
        const float *p = a.part + (2 * k + (k == k0)) * size;
        const float top = p[rows_at_once * D + rr];
        const float f = top == m ? 1.0f : exp2f(top - m);
        l += f * p[rows_at_once * (D + 1) + rr];
        if (D == 128) {
            const float4 y = reinterpret_cast<const float4 *>(p + rr * D)[lane];
            v[0] += f * y.x, v[1] += f * y.y, v[2 % (D / 32)] += f * y.z, v[3 % (D / 32)] += f * y.w;
        } else {
            const float2 y = reinterpret_cast<const float2 *>(p + rr * D)[lane];
            v[0] += f * y.x, v[1] += f * y.y;
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int j = 0; j < D / 32; j += 2) {
        const int64_t at = i * D + lane * (D / 32) + j;
        if (a.out_bf16)
            *reinterpret_cast<__nv_bfloat162 *>(static_cast<uint16_t *>(a.out) + at) =
                __floats2bfloat162_rn(v[j] * inv, v[j + 1] * inv);
        else *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at) = make_float2(v[j] * inv, v[j + 1] * inv);
    }
    if (a.lse && lane == 0) a.lse[i] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
}

// Requests of many rows (attention4_wide.cu).
size_t attention4_wide_workspace(const moe_cache_attn *d, const moe_cache4 *cache);
int launch_attention4_wide(const AttnArgs &args, const moe_cache_attn *d, const moe_cache4 *cache, int few_rows,
                           void *ws, cudaStream_t s);

}  // namespace moe
