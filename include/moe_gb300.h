/*
 * moe_gb300 — the DeepSeek-style Mixture-of-Experts FFN layer at decode time,
 * on one NVIDIA GB300 (sm_103a).
 *
 * The layer (Moreh report "21K output tokens/s DeepSeek inference on MI300X
 * with Expert Parallelism", sections "Overview" and "Parallelisation"):
 * a light gate routes each token to top_k of E small SwiGLU experts, an
 * always-on shared expert runs for every token, and the expert outputs are
 * summed with the routing weights.  Expert-parallel dispatch/combine (the
 * all-to-all of section "Compute-communication overlap") becomes, on one
 * GPU, a permutation of token rows into per-expert contiguous rows and a
 * weighted gather back.
 *
 * Conventions for every call below
 *   - Pointers are DEVICE pointers unless the argument says "host".
 *   - All buffers are allocated by the caller; the library allocates no
 *     memory.  Row-major layouts, innermost dimension last, no padding.
 *     Every device pointer must be 16-byte aligned.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Device calls only enqueue work: none synchronises the host
 *     or reads device data back, and sizes that depend on the routing
 *     (rows per expert) stay on the device, so every device call can be
 *     captured in a CUDA graph (the report's section "Using HIP Graphs":
 *     tensor sizes kept static so that dispatch and combine can live inside
 *     the captured graph).
 *   - Return value: MOE_OK (0) or a negative MOE_ERR_* code.  Argument and
 *     shape errors are returned before anything is enqueued.  Problems only
 *     the device can see (an expert id out of range, inconsistent offsets,
 *     a pipeline wait that ran out of time) set bits MOE_DEV_* in a device
 *     status word (int32) instead; kernels never trap.  `dev_status` may be
 *     NULL (no report).
 *
 * Notation: T tokens, H hidden, I expert intermediate width, E routed
 * experts, S shared experts, k = top_k, G = E + S groups, R = T*k routed
 * rows, R_tot = R + S*T rows.  Groups 0..E-1 are the routed experts in
 * PHYSICAL order, groups E..G-1 the shared experts.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* ---- codes ------------------------------------------------------------ */
enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1,        /* null pointer, bad enum, T < 0, misalignment */
    MOE_ERR_UNSUPPORTED_SHAPE = -2,  /* a dimension this build does not handle */
    MOE_ERR_WORKSPACE_TOO_SMALL = -3,
    MOE_ERR_CUDA = -4,               /* a CUDA runtime call failed */
    MOE_ERR_TIMEOUT = -5,            /* the device reported MOE_DEV_TIMEOUT */
    MOE_ERR_DEVICE_FAULT = -6        /* the device reported another MOE_DEV_* bit */
};
enum {                               /* bits of the device status word */
    MOE_DEV_BAD_EXPERT_ID = 1,       /* a topk id / log2phys entry outside [0, E) */
    MOE_DEV_BAD_OFFSETS = 2,         /* expert_offsets not non-decreasing within [0, rows] */
    MOE_DEV_TIMEOUT = 4,             /* a bounded pipeline wait expired (about 1 s) */
    MOE_DEV_BAD_INDEX = 8,           /* a page, slot, position or length outside its range */
    MOE_DEV_NO_ROOM = 16             /* too few free pages, table columns or token rows */
};
enum { MOE_SCORING_SOFTMAX = 0, MOE_SCORING_SIGMOID = 1 };
enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_FP8_BLOCK128 = 1, MOE_DTYPE_MXFP4 = 2 };  /* MXFP4: moe_layer_few only */
enum { MOE_OUT_F32 = 0, MOE_OUT_BF16 = 1 };
enum { MOE_ACT_IDENTITY = 0, MOE_ACT_SILU_MUL = 1 };
/* Layout of an expert weight tensor W [groups, N, K] (w13, w2):
 *   MOE_LAYOUT_ROWS   row-major, K innermost;
 *   MOE_LAYOUT_TILES  128 x 128-byte tiles, each contiguous, tile-major: tile
 *                     (g, n/128, k/kt) holds rows n%128 of 128 bytes (kt = 128
 *                     e4m3 or 64 bf16 elements), and within row r the 16-byte
 *                     chunk c is stored at chunk position c ^ (r mod 8) (the
 *                     128-byte swizzle the tensor cores read), so a kernel
 *                     places a tile in shared memory with one 16 KB bulk copy.
 * moe_pack_expert_weights converts the first into the second.  Results do
 * not depend on the layout. */
enum { MOE_LAYOUT_ROWS = 0, MOE_LAYOUT_TILES = 1 };

/* ---- layer description -------------------------------------------------- */
typedef struct moe_config {
    int32_t hidden;          /* H; multiple of 128 */
    int32_t inter;           /* I, width of every expert (routed and shared); multiple of 128 */
    int32_t num_experts;     /* E routed experts, 1..1024 */
    int32_t num_shared;      /* S shared experts, 0..4, each of width I */
    int32_t top_k;           /* k, 1..16 */
    int32_t num_groups;      /* expert groups for group-limited routing (1 = none); divides E */
    int32_t topk_groups;     /* groups kept */
    int32_t group_topn;      /* a group's score is the sum of its best group_topn scores */
    int32_t scoring;         /* MOE_SCORING_* */
    int32_t norm_topk;       /* 1: divide the chosen weights by their sum */
    int32_t dtype;           /* MOE_DTYPE_*: weights/activations of the expert GEMMs */
    int32_t max_tokens;      /* largest T the workspace of moe_layer_forward is sized for */
    float routed_scaling;    /* factor on the routed weights (not on shared experts) */
} moe_config;

/* Device pointers to the layer's weights. */
typedef struct moe_weights {
    const void *w_gate;       /* bf16 [E, H], LOGICAL expert order */
    const float *e_bias;      /* fp32 [E] logical, selection-only bias (sigmoid); NULL = none */
    const float *logit_offset;/* fp32 [E] logical, added to the gate logits; NULL = none */
    const int32_t *log2phys;  /* int32 [E]: physical slot of each logical expert (two may share
                                 one); NULL = identity */
    const void *w13;          /* [G, 2I, H]: rows [0, I) gate proj, [I, 2I) up proj; e4m3 or bf16 */
    const float *w13_scales;  /* fp32 [G, 2I/128, H/128], one per 128x128 block (FP8 only) */
    const void *w2;           /* [G, H, I] down proj; e4m3 or bf16 */
    const float *w2_scales;   /* fp32 [G, H/128, I/128] (FP8 only) */
    int32_t expert_layout;    /* MOE_LAYOUT_* of w13 and w2 (scales are always as above) */
} moe_weights;

/* ---- routing -------------------------------------------------------------
 * Gate logits l[t,e] = sum_h x[t,h] Wg[e,h] (+ logit_offset[e]) and top-k
 * selection (report, section "Overview": a light gating network chooses a
 * few experts per token; section "Load balancing across GPUs": after the
 * experts are permuted the gate must emit ids in the new order).
 *   x        bf16 [T, H];  w_gate bf16 [E, H] (logical order)
 *   e_bias   fp32 [E] or NULL (sigmoid scoring only)
 *   logit_offset fp32 [E] or NULL;  log2phys int32 [E] or NULL
 *   logits   fp32 [T, E], written (the gate logits, logical order)
 *   topk_ids int32 [T, k], written: PHYSICAL ids, slot j in descending
 *            selection score (ties: lower logical id first)
 *   topk_w   fp32 [T, k], written: routing weights of the slots
 * Logits are summed in a fixed order (lane-sliced fp32 FMA chains, then a
 * butterfly), so the ids are reproducible bit for bit.  Sigmoid scoring:
 * s = fp32(sigmoid(l)) evaluated in fp64, selection by s + bias, groups
 * scored by the sum of their top group_topn, weights s/sum(s) (x scaling).
 * Softmax scoring: selection by l; weights exp(l - max l) / sum over E (or
 * over the chosen k with norm_topk), each exponential in fp32 of the exact
 * difference, sums and quotient in fp64: within 5.4e-7 (relative) of the
 * fp64 softmax while l - max l > -87. */
MOE_API int moe_route(const moe_config *cfg, int32_t T, const void *x, const void *w_gate,
              const float *e_bias, const float *logit_offset, const int32_t *log2phys,
              float *logits, int32_t *topk_ids, float *topk_w,
              int32_t *dev_status, void *stream);

/* moe_route followed by the FP8 quantisation of x (moe_act_requant with
 * MOE_ACT_IDENTITY) in the launches of moe_route alone: the selection kernel
 * quantises each token's row while the gate logits are computed.  The same
 * results, bit for bit, as the two calls.  FP8 layers only (else
 * MOE_ERR_INVALID_ARG).  xq e4m3 [T, hidden] and xs fp32 [T, hidden/128]
 * (device, caller-owned); other arguments as moe_route.  x must not change
 * until the call's kernels have run (it is read while the logits are
 * computed). */
MOE_API int moe_route_quantize(const moe_config *cfg, int32_t T, const void *x, const void *w_gate,
                               const float *e_bias, const float *logit_offset,
                               const int32_t *log2phys, float *logits, int32_t *topk_ids,
                               float *topk_w, void *xq, float *xs, int32_t *dev_status,
                               void *stream);

/* ---- activation quantisation ----------------------------------------------
 * mode MOE_ACT_IDENTITY (FP8 layers): in bf16 [rows, H] -> out e4m3 [rows, H]
 *   and out_scales fp32 [rows, H/128]: per row and 128-column group,
 *   scale = amax/448 (IEEE fp32 division; 1 if amax = 0),
 *   code = e4m3(v / scale), round to nearest even, saturating.
 * mode MOE_ACT_SILU_MUL: in fp32 [rows, 2I] (gate | up halves), h =
 *   silu(gate) * up in fp32; FP8 layers quantise h as above into
 *   out e4m3 [rows, I] + out_scales [rows, I/128]; BF16 layers write
 *   out bf16 [rows, I] (out_scales unused, may be NULL).
 * rows_dev: NULL, or a device int32 holding the number of rows to process
 *   (clamped to `rows`); e.g. expert_offsets + G.
 * (SGLang/H20 article, section "MoE": the block-scale handling of the MoE
 * GEMMs; the activation format is the R1 FP8 layout, per token x 128.) */
MOE_API int moe_act_requant(const moe_config *cfg, int32_t mode, int32_t rows,
                    const int32_t *rows_dev, const void *in, void *out,
                    float *out_scales, void *stream);

/* ---- dispatch (permutation into per-expert rows) ---------------------------
 * topk_ids int32 [T, k] physical ids.  Routed slot i = t*k + j goes to row
 * expert_offsets[e] + (number of earlier slots with the same expert), so
 * rows of an expert are in increasing slot order (deterministic).  Shared
 * expert s of token t goes to row expert_offsets[E + s] + t.
 *   x_rows     e4m3 [T, H] (FP8) or bf16 [T, H] (BF16): rows to gather
 *   x_scales   fp32 [T, H/128] (FP8 only)
 *   expert_offsets int32 [G + 1], written: first row of every group
 *   src_of_row int32 [R_tot], written: the slot of each row (routed slots
 *              t*k + j; shared slots R + s*T + t)
 *   row_of_slot int32 [T, k], written (-1 for a slot whose id was invalid)
 *   xp         [R_tot, H] gathered rows (e4m3 or bf16), xp_scales fp32
 *              [R_tot, H/128] (FP8 only)
 *   ws         scratch of moe_permute_workspace_size bytes
 *   copy_max_group_rows  the rows of groups with more rows than this get their
 *              src_of_row / row_of_slot entries but are not copied into xp /
 *              xp_scales (a GEMM that gathers them from the token rows,
 *              moe_grouped_gemm_swiglu_gather, reads them there); INT32_MAX
 *              copies every row, < 0 is MOE_ERR_INVALID_ARG.
 * (report, sections "Overview" and "Compute-communication overlap": the
 * dispatch that carries each token to its experts.) */
MOE_API int moe_permute_workspace_size(const moe_config *cfg, int32_t T, size_t *bytes /* host */);
MOE_API int moe_permute(const moe_config *cfg, int32_t T, const int32_t *topk_ids,
                const void *x_rows, const float *x_scales,
                int32_t *expert_offsets, int32_t *src_of_row, int32_t *row_of_slot,
                void *xp, float *xp_scales, void *ws, size_t ws_bytes,
                int32_t copy_max_group_rows, int32_t *dev_status, void *stream);

/* moe_permute without a workspace argument.  The pages have no counterpart:
 * this entry serves callers that cannot allocate device memory, such as a
 * plugin inside a framework that owns every device allocation, or a
 * runtime held to a fixed, pre-reserved memory budget.  Arguments and
 * results are those of moe_permute minus ws/ws_bytes, copying every row.
 *   - Scratch lives in a static device array inside the library, 1 MiB per
 *     device (moe_permute_static_scratch_capacity()), held by every GPU that
 *     loads the library until the process exits.  A call whose scratch need
 *     (moe_permute_workspace_size) exceeds it returns
 *     MOE_ERR_UNSUPPORTED_SHAPE before enqueuing anything; for the R1
 *     shape (256 experts, top 8) that is above 21824 tokens.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.  The address is looked up again when the
 *     device's CUDA context has changed since (after a device reset the
 *     module holding the array is reloaded elsewhere), so the call stays
 *     valid across resets; the first call after a reset should again come
 *     before any capture.
 *   - Every call on a device shares the one array and leaves its contents
 *     behind; nothing in it needs to start at zero (a call reads only words
 *     it wrote earlier).  Calls that overlap on the GPU (other streams, or
 *     concurrent graph branches) race on it: serialise them.
 *   - Allocates nothing: no cudaMalloc, cudaFree or allocating library call. */
MOE_API int moe_permute_static_scratch(const moe_config *cfg, int32_t T, const int32_t *topk_ids,
                                       const void *x_rows, const float *x_scales,
                                       int32_t *expert_offsets, int32_t *src_of_row,
                                       int32_t *row_of_slot, void *xp, float *xp_scales,
                                       int32_t *dev_status, void *stream);
MOE_API size_t moe_permute_static_scratch_capacity(void);

/* ---- group row windows --------------------------------------------------------
 * moe_grouped_gemm, moe_grouped_gemm_swiglu and moe_expert_ffn take a window
 * min_group_rows <= n <= max_group_rows: only the groups whose row count n
 * (expert_offsets[g+1] - expert_offsets[g]) lies in it are computed; the
 * output rows of the other groups are not written.  0 and INT32_MAX select
 * every group; min_group_rows < 0 is MOE_ERR_INVALID_ARG.  A batch can so
 * send its groups of few rows to one kernel and the rest to another: the
 * layer, for wide FP8 batches, runs moe_expert_ffn on the groups of at most
 * 32 rows and the two GEMMs on the others.  Results are bit-identical to a
 * call over every group. */

/* ---- grouped GEMM -----------------------------------------------------------
 * For every group g and row r in [expert_offsets[g], expert_offsets[g+1]):
 *   C[r, n] = sum_k A[r, k] * W[g, n, k]
 * FP8 (cfg->dtype = MOE_DTYPE_FP8_BLOCK128): A e4m3 [rows, K] with a_scales
 *   fp32 [rows, K/128]; W e4m3 [groups, N, K] with w_scales fp32
 *   [groups, N/128, K/128]; every 128-wide K block is scaled by
 *   a_scale[r, kb] * w_scale[g, n/128, kb] (fp32 accumulation).
 * BF16: A bf16 [rows, K], W bf16 [groups, N, K], scales unused.
 * w_layout: MOE_LAYOUT_* of W (else MOE_ERR_INVALID_ARG).
 * C: fp32 or bf16 (c_dtype = MOE_OUT_*) [rows, N]; rows outside every group
 *   are not written.  expert_offsets: device int32 [groups + 1].
 * N multiple of 128; K multiple of 128 and at most 7168 (FP8) or multiple
 * of 64 (BF16); groups <= 1024.
 * Tensor cores (tcgen05, accumulators in tensor memory) fed by TMA; weight
 * rows sit on the MMA's M side and the few token rows of an expert on its
 * N side (the SGLang/H20 article, section "SwapAB GEMM": map the token
 * dimension to the fine-grained side of the MMA for small, variable rows
 * per expert).  FP8 groups averaging 16 rows or more with fp32 C and N a
 * multiple of 256 swap back: 128 token rows on M against 256 output columns
 * on N; same bits. */
MOE_API int moe_grouped_gemm(const moe_config *cfg, int32_t groups, int32_t n_out, int32_t k_dim,
                     int32_t rows, const void *a, const float *a_scales,
                     const int32_t *expert_offsets, const void *w, const float *w_scales,
                     int32_t w_layout, void *c, int32_t c_dtype, int32_t min_group_rows,
                     int32_t max_group_rows, int32_t *dev_status, void *stream);

/* Grouped GEMM with the SwiGLU epilogue (gate/up GEMM and SiLU-mul fused):
 * for the rows r of group g, with W13[g] = [W_gate; W_up] ([2*inter, K]),
 *   g = A[r] W_gate^T, u = A[r] W_up^T (fp32, FP8 block scales as in
 *   moe_grouped_gemm), h = silu(g) * u (fp32), and
 *   FP8 layers: h quantised per row and 128-feature group as in
 *     moe_act_requant -> h e4m3 [rows, inter], h_scales fp32 [rows, inter/128];
 *   BF16 layers: h rounded to bf16 -> h bf16 [rows, inter] (h_scales unused).
 * Gives the same bits as moe_grouped_gemm (fp32 C) followed by
 * moe_act_requant(SILU_MUL), without writing the fp32 gate/up rows.  A tile
 * takes 128 gate rows and the matching 128 up rows, which share one
 * activation tile (the report's "horizontal fusion" of an expert's GEMMs,
 * section "Library optimisation").  FP8 groups averaging 16 rows or more
 * (rows >= 16 * groups) take a second kernel with the orientation swapped:
 * 128 token rows of one expert on the MMA's M side against those 256 weight
 * rows on N, so each thread promotes, applies SwiGLU to and quantises one
 * token row; same bits.  inter multiple of 128; K as in moe_grouped_gemm. */
MOE_API int moe_grouped_gemm_swiglu(const moe_config *cfg, int32_t groups, int32_t inter,
                                    int32_t k_dim, int32_t rows, const void *a,
                                    const float *a_scales, const int32_t *expert_offsets,
                                    const void *w13, const float *w13_scales, int32_t w_layout,
                                    void *h, float *h_scales, int32_t min_group_rows,
                                    int32_t max_group_rows, int32_t *dev_status,
                                    void *stream);

/* moe_grouped_gemm_swiglu without materialised activation rows: the rows of
 * each group are gathered from the token rows of x by the tensor cores' copy
 * engine (TMA tile::gather4, four rows per copy, straight into the MMA's
 * swizzled operand layout), the f1 row gather of the report's fused MoE
 * kernel (section "Library optimisation").  Row r (in expert_offsets' row
 * numbering) is token t(r) of slot src_of_row[r]: routed slots t*top_k + j
 * give t, the shared experts' slots T*top_k + i*T + t give t (moe_permute's
 * tables).  FP8 layers only (else MOE_ERR_INVALID_ARG).
 *   x_rows   e4m3 [T, k_dim] and x_scales fp32 [T, k_dim/128]: the token rows
 *            (moe_route_quantize's xq / xs)
 *   src_of_row int32 [rows]
 * Other arguments, results (h, h_scales rows in dispatch order) and the group
 * row window as moe_grouped_gemm_swiglu, whose token-rows-on-M kernel this is
 * (used for every batch size); the same result bits as that call on the
 * rows moe_permute gathers.  Not the layer's path: each gather4 moves 512
 * bytes, and the 32 of them a 128-row tile needs per 128-byte K block make
 * the copies, not the MMAs or the promotion, set the pace (same box, R1
 * layer: gate/up 1.87 -> 3.72 ms at 4096 tokens, against a 48 us saving in
 * the dispatch). */
MOE_API int moe_grouped_gemm_swiglu_gather(const moe_config *cfg, int32_t groups, int32_t inter,
                                           int32_t k_dim, int32_t rows, const void *x_rows,
                                           const float *x_scales, int32_t T,
                                           const int32_t *src_of_row,
                                           const int32_t *expert_offsets, const void *w13,
                                           const float *w13_scales, int32_t w_layout, void *h,
                                           float *h_scales, int32_t min_group_rows,
                                           int32_t max_group_rows, int32_t *dev_status,
                                           void *stream);

/* ---- the experts' FFN in one kernel ------------------------------------------/* ---- the experts' FFN in one kernel ------------------------------------------
 * For the rows r of every group g (offsets as in moe_grouped_gemm):
 *   g, u = A[r] W13[g]^T     (W13 [groups, 2*inter, hidden], A [rows, hidden];
 *                             FP8: e4m3 with block scales w13_scales fp32
 *                             [groups, 2*inter/128, hidden/128] and a_scales fp32
 *                             [rows, hidden/128]; BF16: bf16, scales unused),
 *   h    = silu(g) * u: FP8 quantised per row and 128-feature group
 *          -> h e4m3 [rows, inter], h_scales fp32 [rows, inter/128];
 *          BF16 rounded -> h bf16 [rows, inter] (h_scales unused),
 *   y[r] = h[r] W2[g]^T      (W2 [groups, hidden, inter], FP8 w2_scales fp32
 *                             [groups, hidden/128, inter/128]) -> y fp32 [rows, hidden].
 * The same bits as moe_grouped_gemm_swiglu followed by moe_grouped_gemm
 * (fp32 C), in one persistent launch: the report's fused MoE kernel
 * (section "Library optimisation") runs an expert's FFN as one kernel.
 * CTAs claim the gate/up tiles, then the down tiles, from a counter; a down
 * tile waits (bounded, about a second, else MOE_DEV_TIMEOUT) until the h
 * rows of its 32-row activation tile are complete, so no wave of either
 * GEMM ends with most of the GPU idle.
 *   sched: device scratch of at least moe_expert_ffn_sched_bytes(groups,
 *   rows) bytes, owned by the caller, cleared by the call on `stream`; one
 *   call at a time per buffer (else MOE_ERR_WORKSPACE_TOO_SMALL if short).
 * cfg supplies dtype, hidden and inter; groups <= 1024 (else
 * MOE_ERR_UNSUPPORTED_SHAPE); a, w13, w2, h and y 16-byte aligned; w_layout
 * the MOE_LAYOUT_* of w13 and w2. */
MOE_API size_t moe_expert_ffn_sched_bytes(int32_t groups, int32_t rows);
MOE_API int moe_expert_ffn(const moe_config *cfg, int32_t groups, int32_t rows, const void *a,
                           const float *a_scales, const int32_t *expert_offsets,
                           const void *w13, const float *w13_scales, const void *w2,
                           const float *w2_scales, int32_t w_layout, void *h,
                           float *h_scales, float *y, int32_t *sched, size_t sched_bytes,
                           int32_t min_group_rows, int32_t max_group_rows,
                           int32_t *dev_status, void *stream);

/* The experts' FFN on dispatched rows with the kernels moe_layer_forward
 * would pick for this batch: moe_expert_ffn for BF16 layers and for FP8
 * groups averaging fewer than 32 rows (rows < 32 * groups); otherwise
 * moe_expert_ffn on the groups of at most 32 rows, then
 * moe_grouped_gemm_swiglu and moe_grouped_gemm (down, fp32 y) on the groups
 * of more (row windows above).  Arguments, layouts, ownership and errors as
 * moe_expert_ffn over every group (sched is cleared on `stream`); every
 * choice gives the same result bits.  Used by the expert-parallel step, where the
 * rows a rank receives for its experts, and its shared-expert rows, are FFN
 * calls of their own. */
MOE_API int moe_experts_forward(const moe_config *cfg, int32_t groups, int32_t rows,
                                const void *a, const float *a_scales,
                                const int32_t *expert_offsets, const void *w13,
                                const float *w13_scales, const void *w2,
                                const float *w2_scales, int32_t w_layout, void *h,
                                float *h_scales, float *y, int32_t *sched, size_t sched_bytes,
                                int32_t *dev_status, void *stream);

/* Packs an expert weight tensor W [groups, n_out, k_dim] (e4m3 for FP8
 * layers, bf16 otherwise, per cfg->dtype) from MOE_LAYOUT_ROWS into
 * MOE_LAYOUT_TILES (w_tiled, same size, device, caller-owned, must not
 * overlap w).  The FFN streams every 128 x 128-byte weight tile as one
 * contiguous 16 KB read instead of 128 rows 7-14 KB apart (a same-box A/B
 * on the R1 decode layer: 1.626 -> 1.560 ms for the one-kernel FFN).
 * n_out multiple of 128; k_dim of 128 (e4m3) or 64 (bf16); 16-byte aligned
 * pointers. */
MOE_API int moe_pack_expert_weights(const moe_config *cfg, int32_t groups, int32_t n_out,
                                    int32_t k_dim, const void *w, void *w_tiled, void *stream);

/* ---- combine -------------------------------------------------------------------
 * out[t, :] = sum_s Y[expert_offsets[E+s] + t, :]
 *           + sum_j topk_w[t, j] * Y[row_of_slot[t, j], :]    (fp32, shared
 * first, then j ascending; slots with row -1 are skipped).
 *   y fp32 [R_tot, H] (the experts' outputs); out fp32 or bf16 [T, H]
 *   (out_dtype = MOE_OUT_*).
 * A gather per token: no atomics, no scatter (report, section "Overview":
 * the combine that brings expert outputs back to their tokens). */
MOE_API int moe_combine(const moe_config *cfg, int32_t T, const void *y, const int32_t *row_of_slot,
                const float *topk_w, const int32_t *expert_offsets, void *out,
                int32_t out_dtype, void *stream);

/* ---- the whole layer -------------------------------------------------------------
 * route (FP8: with the quantisation of x, as moe_route_quantize) -> permute
 * -> the experts' FFN -> combine, all
 * on `stream`.  The experts' FFN is
 *   BF16, and FP8 with groups averaging fewer than 32 rows (decode):
 *     moe_expert_ffn (one persistent kernel);
 *   FP8, groups averaging 32 rows or more: moe_expert_ffn on the groups of
 *     at most 32 rows, then moe_grouped_gemm_swiglu (its token-rows-on-M
 *     kernel) and moe_grouped_gemm down (the same orientation when hidden is
 *     a multiple of 256, else 64-row tiles) on the others;
 * all with the same result bits (fp32 expert outputs), and
 * all intermediates inside `ws` (size from moe_workspace_size for
 * cfg->max_tokens).  x bf16 [T, H]; out fp32 or bf16 [T, H].  T may be 0..
 * max_tokens.  The workspace's device status word is cleared at the start
 * of every call; read it with moe_get_device_status after the stream has
 * finished. */
MOE_API int moe_workspace_size(const moe_config *cfg, size_t *bytes /* host */);
MOE_API int moe_layer_forward(const moe_config *cfg, const moe_weights *w, int32_t T, const void *x,
                      void *out, int32_t out_dtype, void *ws, size_t ws_bytes, void *stream);

/* ---- the whole layer for a few tokens ---------------------------------------------
 * moe_layer_forward's layer for 1 to moe_layer_few_max_tokens() (16) tokens in
 * two kernels: the gate logits (with the quantisation of x), then selection,
 * both expert products and the combine in one persistent kernel that streams
 * each chosen expert's weights once.  The same definition, step by step:
 * routing ids and weights are moe_route's, bit for bit, also with biases of
 * minus infinity (experts taken out); x and h are quantised
 * in the same places (BF16: h is kept to 17 bits instead of rounded to bf16);
 * sums are fp32 in another order, so outputs agree within the layer's tolerance
 * and not bit for bit (a sum that lies on a rounding boundary of h may take the
 * neighbouring code).  Outputs do not depend on
 * timing.
 *   cfg        as for moe_layer_forward, max_tokens 0..16 (else
 *              MOE_ERR_UNSUPPORTED_SHAPE); dtype may also be
 *              MOE_DTYPE_MXFP4: x and h are then quantised to MXFP4 (blocks of
 *              32, below) and w13 / w2 are MXFP4
 *   w          expert_layout must be MOE_LAYOUT_TILES (else
 *              MOE_ERR_INVALID_ARG): w13 and w2 from moe_pack_expert_weights,
 *              with the fp32 block scales in FP8; MXFP4 takes codes and scale
 *              bytes (in the w13_scales / w2_scales pointers) from
 *              moe_mx4_pack_weights
 *   x bf16 [T, H], out fp32 or bf16 [T, H], 0 <= T <= max_tokens
 *   ws         scratch of moe_layer_few_workspace_size bytes, 16-byte aligned,
 *              one call at a time; needs no initialisation
 * A token none of whose choices is valid gets its shared experts alone, or
 * zeros.  The device status word is the first word of ws
 * (moe_get_device_status). */
MOE_API int32_t moe_layer_few_max_tokens(void);
MOE_API int moe_layer_few_workspace_size(const moe_config *cfg, size_t *bytes /* host */);
MOE_API int moe_layer_few(const moe_config *cfg, const moe_weights *w, int32_t T, const void *x,
                          void *out, int32_t out_dtype, void *ws, size_t ws_bytes, void *stream);
/* Byte offsets inside that workspace (host): topk_ids int32 [T, k] (physical,
 * -1 where a choice was invalid) and topk_w fp32 [T, k] are what a caller may
 * want to read; the rest are intermediates. */
typedef struct moe_few_layout {
    size_t status, sched, score, select, topk_ids, topk_w, x, x_scales, h, h_scales, y, total;
} moe_few_layout;
MOE_API int moe_layer_few_layout(const moe_config *cfg, moe_few_layout *layout /* host */);

/* ---- MXFP4 -------------------------------------------------------------------------
 * Microscaled four-bit floating point (OCP MX, e2m1 elements): 32 consecutive
 * elements of a row share a power of two.  With m the block's largest
 * magnitude, e = max(floor(log2 m) - 2, -127) (0 for a block of zeros);
 *   code  = e2m1(v / 2^e), round to nearest even, saturating at 6
 *   scale byte = e + 127.
 * A block holding an infinity or a NaN has the byte 255 and zero codes, and
 * reads back as NaN.
 *   codes  [rows, cols/2] bytes, the even element in the low four bits
 *   scales [rows, cols/32] bytes
 * cols a multiple of 32 (else MOE_ERR_UNSUPPORTED_SHAPE); rows may be 0; in /
 * out fp32 or bf16 (MOE_OUT_*), pointers 16-byte aligned (scales: any). */
MOE_API int moe_mx4_quantize(int32_t rows, int32_t cols, const void *in, int32_t in_dtype,
                             void *codes, void *scales, void *stream);
MOE_API int moe_mx4_dequantize(int32_t rows, int32_t cols, const void *codes, const void *scales,
                               void *out, int32_t out_dtype, void *stream);

/* Expert weights W [groups, n_out, k_dim] in MXFP4, row-major, into the tiles
 * that the products and moe_layer_few read (same sizes, device, caller-owned,
 * no overlap): tile (g, n/128, k/128) holds 128 rows of 64 bytes, 16-byte
 * chunk c of row r at chunk position c ^ ((r/2) mod 4) (the 64-byte swizzle);
 * its 512 scale bytes are at byte (r mod 32)*16 + (r/32)*4 + j for block j of
 * row r, the order the tensor cores take them in.  n_out and k_dim multiples
 * of 128. */
MOE_API int moe_mx4_pack_weights(int32_t groups, int32_t n_out, int32_t k_dim, const void *codes,
                                 const void *scales, void *codes_tiled, void *scales_tiled,
                                 void *stream);

/* Grouped products of MXFP4 rows and MXFP4 weights, as moe_grouped_gemm's:
 * for every group g and row r in [expert_offsets[g], expert_offsets[g+1])
 *   C[r, n] = sum_k A[r, k] W[g, n, k],
 * each operand's value its code times its block's scale, products and sums
 * in fp32 (the tensor cores' four-bit kind; the scales are powers of two).
 *   a, a_scales  codes [rows, k_dim/2] and scale bytes [rows, k_dim/32], as
 *                moe_mx4_quantize gives them
 *   w, w_scales  [groups, n_out, k_dim] in tiles (moe_mx4_pack_weights)
 *   expert_offsets device int32 [groups + 1], as in moe_grouped_gemm; rows
 *                outside every group are not written, a table that is not
 *                non-decreasing within [0, rows] sets MOE_DEV_BAD_OFFSETS and
 *                nothing is computed
 *   c            fp32 or bf16 (MOE_OUT_*) [rows, n_out]
 * n_out and k_dim multiples of 128, groups <= 1024; c (h below) 32-byte
 * aligned, the other pointers 16.
 * The SwiGLU form takes W13 [groups, 2*inter, k_dim] (gate rows, then up rows)
 * and writes h = silu(g) * u, formed in fp32, as MXFP4: codes [rows, inter/2],
 * scale bytes [rows, inter/32]; inter a multiple of 128. */
MOE_API int moe_mx4_grouped_gemm(int32_t groups, int32_t n_out, int32_t k_dim, int32_t rows,
                                 const void *a, const void *a_scales,
                                 const int32_t *expert_offsets, const void *w_tiled,
                                 const void *w_scales_tiled, void *c, int32_t c_dtype,
                                 int32_t *dev_status, void *stream);
MOE_API int moe_mx4_grouped_gemm_swiglu(int32_t groups, int32_t inter, int32_t k_dim, int32_t rows,
                                        const void *a, const void *a_scales,
                                        const int32_t *expert_offsets, const void *w13_tiled,
                                        const void *w13_scales_tiled, void *h, void *h_scales,
                                        int32_t *dev_status, void *stream);

/* ---- norms around a block ------------------------------------------------------------
 * One pass over T rows of `hidden` elements:
 *   n  = w_post ? norm(y) * w_post (+ b_post) : y
 *   r' = residual_scale * residual + branch_scale * gate * n
 *   x  = norm(r') * w_pre (+ b_pre)
 * with norm(v) = v / sqrt(mean(v^2) + eps) (MOE_NORM_RMS) or the same of v -
 * mean(v) (MOE_NORM_LAYER): the norm after a block, its gate and residual
 * scale, and the norm before the next one.  fp32 inside; x is formed from the
 * unrounded r'.
 *   y            [T, hidden] (y_dtype) the block's output, or NULL: r' =
 *                residual_scale * residual (a first pre-norm; gate and w_post
 *                must then be NULL)
 *   residual     [T, hidden] (residual_dtype); residual_out the same type, may
 *                be `residual` itself, or NULL (not written)
 *   gate         by gate_mode: none, [hidden], [T], or [T, hidden]
 *   w_*, b_*, gate  param_dtype; b_* may be NULL; w_post NULL: no post-norm
 *   x_out        bf16 [T, hidden], or NULL (then w_pre, b_pre must be NULL)
 * hidden a multiple of 8, at most 16384; dtypes MOE_OUT_*; eps >= 0; other
 * outputs must not overlap any input. */
enum { MOE_NORM_RMS = 0, MOE_NORM_LAYER = 1 };
enum { MOE_GATE_NONE = 0, MOE_GATE_FEATURE = 1, MOE_GATE_TOKEN = 2, MOE_GATE_FULL = 3 };
typedef struct moe_norm {
    int32_t hidden, kind, y_dtype, residual_dtype, param_dtype, gate_mode;
    float eps, residual_scale, branch_scale;
} moe_norm;
MOE_API int moe_block_norm(const moe_norm *d, int32_t T, const void *y, const void *residual,
                           const void *gate, const void *w_post, const void *b_post,
                           const void *w_pre, const void *b_pre, void *residual_out, void *x_out,
                           void *stream);

/* ---- a cache of keys and values in four bits --------------------------------------------
 * Attention's half of a decoder layer, next to the MoE half above: tables of a
 * paged cache, the norm and rotation of queries and keys with the cache's
 * write, and attention that reads it.
 *
 * The cache holds each token's keys and values of kv_heads heads of `dim`
 * channels in MXFP4 (blocks of 32 channels, as moe_mx4_quantize), in pages of
 * `page` tokens.  Token slot s is row s mod page of page s / page.
 *   codes   [pages, 2, kv_heads, page, dim/2]   (keys, then values)
 *   scales  [pages, 2, kv_heads, page, dim/32]
 * dim 64 or 128; page 16, 32, 64 or 128; kv_heads 1..256; pages * page below
 * 2^31 (byte offsets are 64 bits).  A page's rows that no token was written to
 * may hold anything. */
typedef struct moe_cache4 {
    void *codes, *scales;
    int32_t pages, kv_heads, page, dim;
} moe_cache4;

/* Tables of one step, from the requests' lengths: request b holds held[b]
 * tokens and gets new_tokens[b] more (0: none).  Its page i covers its tokens
 * [i page, (i+1) page); the pages that it lacks are taken from a ring of free
 * ones, request after request.
 *   requests    B, 0..16384
 *   held, new_tokens  int32 [B], >= 0
 *   free_pages  int32 [free_count]: a ring; free_range int64 [2] = {next, end}:
 *               entries next .. end-1 (each mod free_count) are free.  A caller
 *               gives pages back by writing them behind `end`.
 *   table       int32 [B, max_pages], the first ceil(held[b]/page) entries of a
 *               row as earlier steps left them; the new pages' entries are
 *               written, all others left alone
 *   lengths     int32 [B], written: held + new_tokens (may be `held`)
 *   starts      int32 [B+1], written: first token row of each request
 *   slots       int32 [max_tokens], written: the slot of each token row, -1
 *               behind the last one
 *   positions   int32 [max_tokens], written: its position, 0 behind the last
 *   free_out    int64 [2], written: free_range after the step (may be it)
 * A step that cannot be made whole is not made: a negative length or a page
 * id below 0 that a token needs sets MOE_DEV_BAD_INDEX; too few free pages,
 * table columns or token rows MOE_DEV_NO_ROOM; then lengths = held, starts,
 * and positions are 0, slots -1, free_out = free_range and the table is as it
 * was.  (Ids are looked at where tokens join a request's last held page.  A free
 * page whose id is below 0, or so large that its slots pass 32 bits, gives its
 * tokens the slot -2^31, which is in no cache.)  One launch; nothing else may overlap. */
MOE_API int moe_cache_tables(int32_t requests, int32_t page, const int32_t *held,
                             const int32_t *new_tokens, const int32_t *free_pages,
                             int32_t free_count, const int64_t *free_range, int32_t *table,
                             int32_t max_pages, int32_t *lengths, int32_t *starts, int32_t *slots,
                             int32_t *positions, int32_t max_tokens, int64_t *free_out,
                             int32_t *dev_status, void *stream);

/* Norm of queries and keys for each head and the rotation by the token's
 * position, in one pass, with the cache's write: for each head v of a row
 *   n = v / sqrt(mean(v^2) + eps) * w           (v itself without w)
 * and the first rope_dim channels of n turned by the token's angles,
 *   MOE_ROPE_HALVES  channels i and i + rope_dim/2 as a pair (i < rope_dim/2)
 *   MOE_ROPE_PAIRS   channels 2i and 2i + 1
 *   a, b -> a cos_i - b sin_i, b cos_i + a sin_i
 * fp32 from load to store, each output rounded once; cached keys have the codes
 * of exact values (as fp64 would give them; sums of squares are fp32 numbers all
 * the same, values of 2^60 and more may pass them).
 *   qkv         bf16 [T, qkv_stride]: q_heads, then kv_heads of keys, then
 *               kv_heads of values, `dim` channels each (dim 64 or 128;
 *               qkv_stride a multiple of 8)
 *   positions   int32 [T]; cos_sin fp32 [max_positions, rope_dim]: cosines of
 *               the rope_dim/2 angles, then sines; both may be NULL with rope_dim 0
 *   w_q, w_k    [dim] of param_dtype (MOE_OUT_*), or NULL
 *   q_out       bf16 [T, q_heads, dim]; k_out bf16 [T, kv_heads, dim] or NULL
 *   cache, slots  NULL, or the keys (after all this) and the values of row t
 *               go to slot slots[t] (int32 [T]; -1: nowhere), in four bits.
 *               Slots of one call are distinct.
 * rope_dim a multiple of 16, 0..dim.  A position outside [0, max_positions) or a
 * slot outside [-1, pages * page) sets MOE_DEV_BAD_INDEX; of such a row nothing
 * is written.  Outputs must not overlap inputs. */
enum { MOE_ROPE_HALVES = 0, MOE_ROPE_PAIRS = 1 };
typedef struct moe_qk_rope {
    int32_t q_heads, kv_heads, dim, rope_dim, style, param_dtype, max_positions, qkv_stride;
    float eps;
} moe_qk_rope;
MOE_API int moe_qk_norm_rope(const moe_qk_rope *d, int32_t T, const void *qkv,
                             const int32_t *positions, const float *cos_sin, const void *w_q,
                             const void *w_k, void *q_out, void *k_out, const moe_cache4 *cache,
                             const int32_t *slots, int32_t *dev_status, void *stream);

/* The values that n slots of a cache hold: k, v bf16 [n, kv_heads, dim] (either
 * may be NULL).  Rows of slot -1 are left as they were; other slots outside
 * the cache set MOE_DEV_BAD_INDEX and leave theirs too. */
MOE_API int moe_cache_read(const moe_cache4 *cache, int32_t n, const int32_t *slots, void *k, void *v,
                           int32_t *dev_status, void *stream);

/* Attention over the cache.  Request b's query rows are starts[b] ..
 * starts[b+1]-1 of q, its last tokens: row i of n stands at position
 * p = lengths[b] - n + i and sees the cached tokens j <= p (with a window,
 * j > p - window):
 *   o = sum_j softmax_j(scale q . k_j) v_j
 * for each query head, with keys and values of KV head
 * head / (q_heads / kv_heads); decode steps, drafted tokens and chunks of
 * prompts in one call.
 *   q, out     bf16 [rows, q_heads, dim] (out may be q); out fp32 with out_dtype
 *              MOE_OUT_F32
 *   lse        fp32 [rows, q_heads] or NULL: the natural logarithm of
 *              sum_j exp(scale q . k_j)
 *   table      int32 [requests, max_pages]; lengths int32 [requests];
 *              starts int32 [requests + 1] (moe_cache_tables' outputs)
 * A row that sees nothing (its position is negative), or only scores of -infinity,
 * gets zeros and an lse of -infinity.  Rows outside every request are left as they were.  starts that
 * decrease or leave [0, rows], lengths outside [0, max_pages * page] and page
 * ids outside [0, pages) set MOE_DEV_BAD_INDEX: such a request is not computed,
 * the tokens of such a page are not seen.
 * Scores and sums are fp32; probabilities are rounded to fp16 before the sum of
 * the values: each is off by 2^-11 of itself at most, or by 2^-36 of the row's
 * largest where that is more (2^-30 where max_q query tokens are more than 32
 * rows, query tokens times heads of a KV head).  Keys and values count
 * whatever their size, up to 2^95 (sums may overflow beyond; a key block whose scale byte is 0,
 * 2^-127, may count as zero): nothing that a row does not see changes its result.
 *   desc.max_q    the most query tokens of one request: what the kernels and the
 *                 workspace are chosen by.  With more than 32 rows the kernels for
 *                 many rows are launched too, also for a step that has none for them.
 *                 Requests of more are computed all the same (slowly, where max_q says that
 *                 there are few), unless their units of work (128 tokens by 8
 *                 rows and more) pass 2^30 / requests: MOE_DEV_BAD_INDEX, and not computed
 *   desc.max_len  the longest request; has to be 0 or more, nothing is chosen by it
 *   ws         moe_cache_attention_workspace_size bytes, 16-byte aligned; one call
 *              at a time; needs no initialisation
 * requests 0..4096, rows * q_heads below 2^31, q_heads a multiple of kv_heads. */
typedef struct moe_cache_attn {
    int32_t requests, rows, q_heads, max_pages, max_q, max_len, window;   /* window 0: none */
    float scale;
} moe_cache_attn;
MOE_API int moe_cache_attention_workspace_size(const moe_cache_attn *d, const moe_cache4 *cache,
                                               size_t *bytes /* host */);
MOE_API int moe_cache_attention(const moe_cache_attn *d, const moe_cache4 *cache, const void *q,
                                const int32_t *table, const int32_t *lengths, const int32_t *starts,
                                void *out, int32_t out_dtype, float *lse, void *ws, size_t ws_bytes,
                                int32_t *dev_status, void *stream);

/* Products of 1 to 16 rows with weights in four bits and activations in bf16:
 *   y[t, n] = sum_k x[t, k] W[n, k],   y fp32 or bf16 [T, n_out] (out_dtype)
 *   MOE_W4_MX   W in MXFP4: codes [n_out, k_dim/2] and scale bytes
 *               [n_out, k_dim/32] as moe_mx4_quantize gives them (row-major)
 *   MOE_W4_INT  W[n, k] = scale[n, k/group] (code - zero[n, k/group]), codes 0..15
 *               (even k in the low four bits), scales bf16 or fp32 (scale_dtype),
 *               zero points uint8 0..15 or NULL (8); group 32, 64 or 128
 * fp32 accumulation; weights up to 2^96 (sums may overflow beyond), scale byte 0 (2^-127)
 * counts as zero.  x is taken as fp16 times a power of two for each row
 * (and part of K): each value is off by 2^-29 of a row's largest at most.  n_out up to 2^30, k_dim a multiple of
 * the group (of 32 for MXFP4), at most 32768; x and codes 16-byte aligned. */
enum { MOE_W4_MX = 0, MOE_W4_INT = 1 };
typedef struct moe_w4 {
    int32_t n_out, k_dim, kind, group, scale_dtype;
} moe_w4;
MOE_API int moe_w4_matvec(const moe_w4 *d, int32_t T, const void *x, const void *codes,
                          const void *scales, const void *zeros, void *y, int32_t out_dtype,
                          void *stream);

/* Byte offsets of the intermediates inside the layer workspace (host), for
 * callers that want to read routing results or rows per expert.  gate_up is
 * an empty region (no layer path keeps fp32 gate/up rows); it stays for
 * layout compatibility. */
typedef struct moe_ws_layout {
    size_t status, logits, topk_ids, topk_w, xq, xs, expert_offsets, src_of_row,
        row_of_slot, perm_scratch, xp, xp_scales, gate_up, h, h_scales, y, ffn_sched, total;
} moe_ws_layout;
MOE_API int moe_workspace_layout(const moe_config *cfg, moe_ws_layout *layout /* host */);

/* Synchronously reads the status word of a layer workspace (device) into
 * *status (host).  Returns MOE_OK when no bit is set, MOE_ERR_TIMEOUT when
 * MOE_DEV_TIMEOUT is set, MOE_ERR_DEVICE_FAULT for any other bit. */
MOE_API int moe_get_device_status(const void *ws, int32_t *status /* host */);

/* Static text for a MOE_OK / MOE_ERR_* code. */
MOE_API const char *moe_status_string(int32_t code);

/* What the last call on this host thread that returned MOE_ERR_CUDA failed
 * at: the CUDA runtime or driver call and its error text (e.g.
 * "cudaLaunchKernelEx: too many resources requested for launch").  Empty
 * until such a failure; a later successful call does not clear it.  The
 * pointer stays valid for the thread's lifetime. */
MOE_API const char *moe_last_error_detail(void);

/* Number of kernels moe_layer_forward enqueues for this configuration. */
MOE_API int moe_layer_kernel_count(const moe_config *cfg, int32_t T);

/* Measurement utility (no counterpart on the pages): streams `bytes` of device
 * memory at `src` through shared memory and discards them, so that the time
 * of the call (timed by the caller with events on `stream`) gives this GPU's
 * read-only HBM rate -- the denominator for kernels bound by streaming
 * weights, which a copy (read + write) figure understates.  One CTA per SM,
 * 64 KB bulk copies, a 3-deep ring.  src 16-byte aligned; bytes a multiple
 * of moe_stream_read_granule() (else MOE_ERR_INVALID_ARG); nothing is written
 * to global memory.  A bounded wait that expires sets MOE_DEV_TIMEOUT in
 * *dev_status (may be NULL). */
MOE_API size_t moe_stream_read_granule(void);
MOE_API int moe_stream_read(const void *src, size_t bytes, int32_t *dev_status, void *stream);

/* Self-test of the bounded waits (no counterpart on the pages: a robustness
 * check of this library).  Launches one warp that waits on a completed
 * mbarrier (must succeed) and on one nothing arrives on (must give up after
 * limit_ns, 1e3..1e8, setting MOE_DEV_TIMEOUT in *dev_status).  Writes
 * *dev_result = 1 (first wait passed) | 2 (second wait gave up).  The
 * kernel always returns; nothing traps. */
MOE_API int moe_selftest_bounded_wait(int32_t *dev_status, int64_t limit_ns, int32_t *dev_result,
                                      void *stream);

/* Self-test of the routing's sigmoid score (csrc/numerics.cuh sigmoid_score):
 * for i < n, fast[i] is the score as the selection kernel computes it (fp32
 * double-float arithmetic, the fp64 expression where that cannot decide the
 * rounding) and ref[i] = fp32(1 / (1 + exp(-logits[i]))) evaluated in fp64;
 * the two must be equal bit for bit.  *fallbacks (device int32, zeroed by the
 * caller) is incremented once per value that took the fp64 evaluation.  All
 * pointers are device pointers of n elements owned by the caller; the call is
 * asynchronous on `stream`.  MOE_ERR_INVALID_ARG: n < 0 or a null pointer. */
MOE_API int moe_selftest_sigmoid(const float *logits, int32_t n, float *fast, float *ref,
                                 int32_t *fallbacks, void *stream);

/* Self-test of moe_expert_ffn's inter-CTA wait (no counterpart on the pages:
 * a robustness check of this library).  Runs the one-kernel FFN on a tiny
 * problem (hidden 128, inter 256, one group, one row) whose scheduler
 * counter starts past the gate/up units, so the down unit waits for h rows
 * that no CTA will write: its bounded wait gives up after about a second,
 * sets MOE_DEV_TIMEOUT in *dev_status, and every CTA drains its copies and
 * MMAs, frees its tensor memory and exits; nothing traps and the context
 * stays usable.  scratch: device, 16-byte aligned, at least
 * moe_selftest_ffn_flag_timeout_scratch_bytes() bytes, owned by the caller
 * (cleared by the call). */
MOE_API size_t moe_selftest_ffn_flag_timeout_scratch_bytes(void);
MOE_API int moe_selftest_ffn_flag_timeout(void *scratch, size_t scratch_bytes,
                                          int32_t *dev_status, void *stream);

/* ---- continuous load balancing ------------------------------------------------
 * Report, section "Load balancing across GPUs": in serving, activation
 * frequencies are re-measured periodically and a new expert permutation is
 * generated from them.
 * moe_count_expert_rows: counts[p] += expert_offsets[p+1] - expert_offsets[p]
 *   for every routed expert p (PHYSICAL order), i.e. this batch's rows per
 *   expert; counts is a device int64 [E] accumulator owned by the caller.
 *   Exact integer sums: the result does not depend on launch order.
 * moe_relayout_experts: dst block p = src block src_slot[p] for p < groups,
 *   each block block_bytes long (a multiple of 16; e.g. one expert's W13,
 *   W2 or scales).  src_slot is a device int32 [groups] table; an entry
 *   outside [0, groups) copies nothing and sets MOE_DEV_BAD_EXPERT_ID in
 *   *dev_status (nullable).  src and dst must not overlap (checked).
 *   Applying a new permutation: with old/new logical->physical tables,
 *   src_slot[p] = old_log2phys[new_phys2log[p]] for routed p, and p itself for
 *   the shared experts; run it on a side stream into second buffers while the
 *   layer keeps serving, then switch pointers. */
MOE_API int moe_count_expert_rows(const moe_config *cfg, const int32_t *expert_offsets,
                                  int64_t *counts, void *stream);
/* SGLang/H20 article, section "Expert Affinity EPLB": track which experts a
 * token selects together.  coact[a*E + b] += 1 for every token of the
 * batch and every two of its k selected experts a != b, as LOGICAL ids
 * (topk_ids are physical; phys2log, device int32 [E], maps them back;
 * NULL = identity).  coact: device int64 [E, E] accumulator, symmetric.
 * Integer atomics: the sums do not depend on order.  Ids out of range are
 * skipped. */
MOE_API int moe_count_coactivation(const moe_config *cfg, int32_t T, const int32_t *topk_ids,
                                   const int32_t *phys2log, int64_t *coact, void *stream);
MOE_API int moe_relayout_experts(const void *src, void *dst, const int32_t *src_slot,
                                 int32_t groups, int64_t block_bytes, int32_t *dev_status,
                                 void *stream);

/* ---- host: balanced expert permutation ----------------------------------------------
 * Report, section "Load balancing across GPUs": from measured activation
 * counts, group the E experts into num_sets sets of E/num_sets with totals
 * as even as possible (a variant of balanced number partitioning) and
 * renumber them so each set is contiguous.  Objective: minimise the largest
 * set total.  Exact (branch and bound) when E <= 16, otherwise
 * cardinality-constrained greedy (largest first into the lightest open set)
 * followed by improving pairwise swaps.  Set s holds physical ids
 * [s*m, (s+1)*m), m = E/num_sets, logical ids ascending inside a set.
 *   counts    host int64 [E], >= 0
 *   log2phys  host int32 [E], written; phys2log host int32 [E], written
 *   max_over_mean host, written (may be NULL): largest set total / mean
 * Pure host code; usable without a GPU. */
MOE_API int expert_balance_permutation(const int64_t *counts, int32_t num_experts, int32_t num_sets,
                               int32_t *log2phys, int32_t *phys2log, double *max_over_mean);

/* Host: the set imbalance of a given permutation (the figure the report,
 * section "Load balancing across GPUs", quotes: the busiest set against the
 * average).  Set s holds physical ids [s*m, (s+1)*m), m = E/num_sets; the
 * load of a set is the sum of counts[e] over the logical experts e with
 * log2phys[e] in it.
 *   counts    host int64 [E], >= 0
 *   log2phys  host int32 [E], a permutation of 0..E-1 (NULL = identity)
 *   max_over_mean host, written: largest set load / mean set load (1 when
 *             every count is 0)
 * MOE_ERR_INVALID_ARG for a negative count, an id out of range or repeated,
 * or E not a multiple of num_sets.  Pure host code; usable without a GPU. */
MOE_API int expert_set_imbalance(const int64_t *counts, const int32_t *log2phys,
                                 int32_t num_experts, int32_t num_sets, double *max_over_mean);

/* Host: affinity-aware placement (SGLang/H20 article, section "Expert
 * Affinity EPLB").  From per-expert counts and the symmetric co-activation
 * matrix coact (host int64 [E, E]), group the experts into num_sets equal
 * sets that keep as much co-activation inside sets as possible while every
 * set total stays within max(L*, floor((1 + load_slack) * mean)), L* being
 * the largest set total of the balanced partition above.  Exact for
 * E <= 16, otherwise best-improvement swaps from the balanced partition.
 * Same layout rule and outputs as expert_balance_permutation, plus
 * *intra_fraction (nullable): co-activation kept inside sets / all of it. */
MOE_API int expert_affinity_permutation(const int64_t *counts, const int64_t *coact,
                                        int32_t num_experts, int32_t num_sets, double load_slack,
                                        int32_t *log2phys, int32_t *phys2log,
                                        double *max_over_mean, double *intra_fraction);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_H */
