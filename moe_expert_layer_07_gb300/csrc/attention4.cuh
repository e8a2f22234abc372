// What the attention kernels over the four-bit cache share: the work list of a
// call, and where the results of a piece of a request are kept.
#pragma once

#include <stdint.h>

#include "internal.h"

namespace moe {

constexpr int kAttnMaxRequests = 4096;
constexpr int kAttnTile = 16;      // tokens of a tile
constexpr int kAttnWarps = 8;
constexpr int kAttnChunk = kAttnTile * kAttnWarps;   // tokens of a unit of work

// Probabilities are 2^(score - ref), fp16 in the products.  They may be up to 2^kAttnTop; where one passes
// that, ref rises so that the largest is 2^11 (few rows) or 2^7 (many).  fp16 has all of its bits down to
// 2^-14, 2^-25 and 2^-21 of the row's largest, and some down to 2^-24.  (With the largest at 2^0 tokens of
// 2^-14 lost bits and of 2^-25 were gone: all of the result where the largest one's value is zero.)
// Eleven bits of P are what one product with fp16 values takes; the rest as a second number would double the
// products of values.  bf16 results do not show it: they and those of fp32 probabilities are 1.6e-3 from fp64's.
constexpr float kAttnTop = 15.0f;

// What a CTA began and others went on with: `nrows` rows (0: nothing) from row rowbase
// of a request whose query rows begin at row0, of the heads from head0, as far as CTA
// `last`.
struct AttnCut {
    int row0, head0, rowbase, nrows, last, pad[3];
};

struct AttnArgs {
    const uint16_t *q;
    const uint8_t *codes, *scales;
    const int32_t *table, *lengths, *starts;
    void *out;
    float *lse;
    int32_t *status;
    // partial results, two to a CTA: weighted sums [rows, D], then ref and sum of each row
    float *part;
    AttnCut *cuts;   // [CTAs]
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

// Joins the rows that were cut between CTAs: `rows_at_once` rows to a partial result,
// `ctas` CTAs in the kernel that left them.
int launch_attention4_join(const AttnArgs &a, int dim, int rows_at_once, int ctas, cudaStream_t s);

// Requests of many rows (attention4_wide.cu).
size_t attention4_wide_workspace(const moe_cache_attn *d, const moe_cache4 *cache);
int launch_attention4_wide(const AttnArgs &args, const moe_cache_attn *d, const moe_cache4 *cache, int few_rows,
                           void *ws, cudaStream_t s);

}  // namespace moe
