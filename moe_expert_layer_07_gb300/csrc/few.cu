// The whole MoE layer for a few tokens (1 to 16) in two kernels.
//
//  few_route_kernel  gate logits in the summation order of moe_route (lane L of
//                    a warp sums the 16-byte chunks L, L+32, ... of the hidden
//                    dimension with fp32 FMA, then a butterfly: the same bits),
//                    the quantisation of x, and the zeroing of the counters.
//  few_ffn_kernel    one persistent CTA per SM: expert selection (every CTA
//                    for itself, no exchange), the experts' gate/up products
//                    with SwiGLU, their down products, and the combine.
//
// With so few rows an expert's weights are read for one to a few products
// each, so the time is the weights' bytes over the memory rate: 400 MB, 59 us
// at the copy rate, for one token of nine 44 MB experts in FP8, where the two
// kernels take 69 to 73 (graph replays 69.2 / 70.9 / 71.2 on three GPUs, calls
// from Python in a row 73.2).  The difference is the first kernel and the selection
// (about 8 us, in which only the shared experts' weights move, to L2) and the
// join of the two phases.  In the FFN kernel everything hides behind the
// stream of weights; its warps are:
//   producer   keeps a ring of weight tiles (MOE_LAYOUT_TILES, bulk copies)
//              full, and runs ahead into the next unit, and into the down
//              products, while the tokens still wait for h
//   tokens     the other side of the products, x or h, into the same stages
//   consumers  the products
//   publishers a unit's results to h or y, and the combine, while the
//              consumers are in the next unit
//
// Units, claimed in order from a counter: for every active group (an expert
// with rows) and 128 of its features, gate and up (2 x 128 weight rows against
// the group's token rows; h = silu(g) u, rounded or quantised, to global
// memory); then for every active group and 128 hidden columns, down.  A down
// unit waits (bounded) until its group's h is complete.  Every unit that is
// waited for was claimed before by a running CTA, which finishes it without
// waiting for anyone, so no co-residency is assumed.  The warp that adds the
// last group's rows to 32 columns combines them for all tokens, in the combine
// kernel's order: no atomic sums, the result does not depend on who came when.
//
// BF16 and FP8 products use the warp-wide MMA (m16n8): 16 weight rows of a warp
// on its M side, up to 8 tokens on N.  tcgen05 would leave its 128-row tile's
// accumulators to be read back and scaled per 128 of K in FP8; here they are
// already in registers, and the tensor rate does not matter: at 24 bytes of
// weights a clock and SM the warps' MMA is under a quarter busy.  A thread
// reads 16 bytes of a weight row at a time (the order of K inside a product is
// free as long as both sides agree), rows 0, 4, 1, 5, ... of eight in MMA
// order, which makes the reads conflict-free on the swizzled tiles.  MXFP4
// carries twice the values per byte, whose conversion kept the warps busy for
// longer than the bytes took to come; there one thread issues tcgen05's
// block-scaled products, which take codes and scales as they are.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "internal.h"
#include "mx4.cuh"
#include "numerics.cuh"
#include "ptx.cuh"
#include "route_select.cuh"
#include "tma_host.h"

namespace moe {
namespace {

constexpr int kMaxT = kFewMaxTokens;
constexpr int kMaxShared = 4;
constexpr int kMaxSlots = kMaxT * 16;                   // routed slots
constexpr int kMaxRows = kMaxSlots + kMaxT * kMaxShared;
constexpr int kMaxGroups = kMaxSlots + kMaxShared;      // groups with rows, each at most 8 NT

enum { DT_BF16 = MOE_DTYPE_BF16, DT_FP8 = MOE_DTYPE_FP8_BLOCK128, DT_MX4 = MOE_DTYPE_MXFP4 };

// The token side, x and h.
//  BF16   x's rows as they are; h in two bf16 parts, h = hi + lo to 17 bits, 64
//         values of hi and then of lo: the products run twice over the same
//         weights, which are what the time goes into.  (One part, as the large
//         batches' kernel keeps, made the output's error 2.3e-3 where its own
//         rounding to bf16 makes 1.7e-3.)
//  FP8    segments of 128 values of a row: each code kept as the fp16 number it
//         stands for before its scale (256 bytes), then the fp32 scale.  Such a
//         segment is one bulk copy.
//  MXFP4  packed codes, row-major; scale bytes as [K tile][row][16] with a
//         row's four of the tile in front: tile and row as the boxes of codes,
//         16 rows from any row one bulk copy (which wants its start aligned).
constexpr int kSegment = 272;
constexpr int kScaleRow = 16;

struct FewArgs {
    int T, H, I, E, S, k, out_bf16;
    const uint8_t *w13, *w2;
    const void *w13_s, *w2_s;
    const float *score, *select;   // [T, E]
    int32_t *ids;
    float *wts;
    const uint8_t *xrows;          // bf16 [T, H], or segments [T, H/128] (FP8)
    uint8_t *hrows;                // [rows, I/64][hi, lo][64] (BF16), segments [rows, I/128], or codes [rows, I/2]
    const uint8_t *xs;             // MXFP4: [H/128][16][kScaleRow]
    uint8_t *hs;                   // MXFP4: [I/128][hs_rows][kScaleRow]
    int hs_rows;
    size_t pf_w13, pf_w2, pf_w13_one, pf_w2_one;   // bytes to prefetch; of one expert
    float *y;                      // [rows, H]
    void *out;
    int32_t *sched;                // unit counter | h_done[kMaxGroups] | col_done[H/128][kPublishers]
    int32_t *status;
};

// ---- kernel 1 ---------------------------------------------------------------

constexpr int kRouteThreads = 128;
constexpr int kTokChunk = 4;   // tokens a warp takes against one gate row

struct RouteArgs {
    int T, H, E, sched_ints, logit_blocks, dtype;
    const uint16_t *x, *wg;
    const float *offset;
    SelectArgs sel;
    float *score, *select;   // [T, E]: SelectArgs' scores (softmax: logits), what it compares
    uint8_t *xq, *xs;
    int32_t *sched, *status;
};

__device__ __forceinline__ void bf8(const uint4 &a, float (&f)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}

// The logits of gate row `w` with NT token rows of x.
template <int NT>
__device__ __forceinline__ void gate_dots(const uint16_t *w, const uint16_t *x, int H, int lane,
                                          float (&acc)[kTokChunk]) {
    // Chunks of each row under way.  More of them make the code longer, and cold
    // instructions cost more than the loads save: 14 for one token was 0.5 us
    // slower, all 28 of the gate row 3 us.
    constexpr int U = 7;
    const int n8 = H / 8;
    for (int c0 = lane; c0 < n8; c0 += 32 * U) {
        uint4 wv[U], xv[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + 32 * u;
            if (c >= n8) continue;
            wv[u] = __ldg(reinterpret_cast<const uint4 *>(w) + c);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                xv[u][t] = __ldg(reinterpret_cast<const uint4 *>(x + (size_t)t * H) + c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c0 + 32 * u >= n8) continue;
            float wf[8];
            bf8(wv[u], wf);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float xf[8];
                bf8(xv[u][t], xf);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[t] = fmaf(xf[j], wf[j], acc[t]);
            }
        }
    }
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) {
    return *reinterpret_cast<uint32_t *>(&h);
}

// fp16 values of the e4m3 codes of four values times or over a scale
__device__ __forceinline__ uint2 fp8_as_half4(float a, float b, float c, float d) {
    const __nv_fp8x2_storage_t lo =
        __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi =
        __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    const __half2_raw l = __nv_cvt_fp8x2_to_halfraw2(lo, __NV_E4M3);
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(hi, __NV_E4M3);
    return make_uint2(half2_bits(__half2(l)), half2_bits(__half2(h)));
}

// One 256-column segment of a token's row, quantised as the layer does
// (quant_row_segment's arithmetic, or mx4.cu's).
__device__ __forceinline__ void quant_segment(const RouteArgs &a, int t, int seg, int lane) {
    const int col = seg * 256 + lane * 8;
    const bool active = col < a.H;
    float f[8] = {};
    if (active) bf8(__ldg(reinterpret_cast<const uint4 *>(a.x + (size_t)t * a.H + col)), f);
    if (a.dtype == DT_FP8) {
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
#pragma unroll
        for (int s = 8; s >= 1; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
        const float sc = fp8_group_scale(amax);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __fdiv_rn(f[j], sc);
        const uint2 p = fp8_as_half4(f[0], f[1], f[2], f[3]), q = fp8_as_half4(f[4], f[5], f[6], f[7]);
        uint8_t *at = a.xq + ((size_t)t * (a.H / 128) + col / 128) * kSegment;
        if (active) *reinterpret_cast<uint4 *>(at + col % 128 * 2) = make_uint4(p.x, p.y, q.x, q.y);
        if (active && (lane & 15) == 0) *reinterpret_cast<float *>(at + 256) = sc;
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t byte = mx4_scale_byte(m);
        if (active) *reinterpret_cast<uint32_t *>(a.xq + ((size_t)t * a.H + col) / 2) = mx4_codes8(f, byte);
        if (active && (lane & 3) == 0)
            a.xs[((size_t)(col / 128) * kMaxT + t) * kScaleRow + col % 128 / 32] = (uint8_t)byte;
    }
}

__global__ void __launch_bounds__(kRouteThreads) few_route_kernel(const RouteArgs a) {
    ptx::pdl_launch_dependents();
    const int gtid = blockIdx.x * kRouteThreads + threadIdx.x, nthreads = gridDim.x * kRouteThreads;
    const int lane = threadIdx.x & 31, warp = gtid >> 5;
    const int chunks = (a.T + kTokChunk - 1) / kTokChunk;
    const int e = warp / chunks, t0 = warp % chunks * kTokChunk;
    ptx::pdl_wait();   // x, and the last call's use of the workspace
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    for (int i = gtid; i < a.sched_ints; i += nthreads) a.sched[i] = 0;
    if ((int)blockIdx.x >= a.logit_blocks) {
        const int q = warp - a.logit_blocks * (kRouteThreads / 32), segs = (a.H + 255) / 256;
        if (q < a.T * segs) quant_segment(a, q / segs, q % segs, lane);
        return;
    }
    if (e >= a.E) return;
    const int nt = min(kTokChunk, a.T - t0);
    const uint16_t *w = a.wg + (size_t)e * a.H, *x = a.x + (size_t)t0 * a.H;
    float acc[kTokChunk] = {};
    if (nt == 1) gate_dots<1>(w, x, a.H, lane, acc);
    else if (nt == 2) gate_dots<2>(w, x, a.H, lane, acc);
    else if (nt == 3) gate_dots<3>(w, x, a.H, lane, acc);
    else gate_dots<4>(w, x, a.H, lane, acc);
#pragma unroll
    for (int t = 0; t < kTokChunk; ++t) {
        float v = acc[t];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (lane == t) acc[0] = a.offset ? __fadd_rn(v, a.offset[e]) : v;
    }
    if (lane < nt) {
        const size_t at = (size_t)(t0 + lane) * a.E + e;
        float s, c;
        expert_scores(a.sel, e, true, acc[0], s, c);
        a.score[at] = s;
        a.select[at] = c;
    }
}

// ---- kernel 2 ---------------------------------------------------------------

constexpr int kConsumers = 8;     // warps that multiply: 16 weight rows of a tile each
constexpr int kProducer = kConsumers, kTokens = kProducer + 1, kFirstPublisher = kTokens + 1;
constexpr int kPublishers = 4;
constexpr int kWarps = kFirstPublisher + kPublishers;
constexpr int kFfnThreads = kWarps * 32;
constexpr int kUnitSlots = 8;     // units announced ahead
constexpr int kPrefetchBytes = 8192;
// The shared experts' part of W13 and of W2 that is fetched ahead, far inside
// L2 (one token of the 256-expert layer: 76.8 us without, 74.7 with 12 MB,
// 75.0 with 24; three with MXFP4 experts 102 / 100.4 / 100.7).
constexpr size_t kPrefetchMost = 24u << 20;

template <int DT, int NT>
struct Traits {
    // K elements of one tile, bytes of its codes; a stage holds two tiles
    static constexpr int kKT = DT == DT_BF16 ? 64 : 128;
    static constexpr int kTile = 16384;
    // the token side of one tile of K: 8 NT rows.  The pitch spreads the reads
    // of a quarter warp (two rows, four chunks each) over all banks.
    static constexpr int kCopyX = DT == DT_BF16 ? 128 : kSegment;   // of one row of x, of h
    static constexpr int kCopyH = DT == DT_BF16 ? 256 : kSegment;
    static constexpr int kPitch = DT == DT_BF16 ? 320 : 272;
    static constexpr int kTokOff = 2 * kTile;
    static constexpr int kTokHalf = 8 * NT * kPitch;
    static constexpr int kWsOff = kTokOff + 2 * kTokHalf;   // FP8: the tiles' two scales
    static constexpr int kStage = (kWsOff + 16 + 127) / 128 * 128;
    static constexpr int kBWords = DT == DT_BF16 ? 8 : 16;  // B words a lane holds for a tile
    static constexpr int kTiles = 2, kScale = 0;
    static constexpr int kMultipliers = kConsumers;         // warps that release a stage
    static constexpr int kReaders = kWarps - 1;             // warps that read a unit's number
};
template <int NT>
struct Traits<DT_MX4, NT> {
    static constexpr int kKT = 128;
    static constexpr int kTile = 8192, kScale = 512;
    static constexpr int kTiles = 4;                        // two of gate and of up, or four of W2
    static constexpr int kTokBytes = 16 * 64, kTokScale = 16 * kScaleRow;
    static constexpr int kTokOff = kTiles * kTile, kScaleOff = kTokOff + kTiles * kTokBytes;
    static constexpr int kTokScaleOff = kScaleOff + kTiles * kScale;
    static constexpr int kStage = kTokScaleOff + kTiles * 512;
    static constexpr int kCopyX = 0, kCopyH = 0, kPitch = 0, kTokHalf = 0, kWsOff = 0;
    static constexpr int kMultipliers = 1;                  // the MMAs' commit
    static constexpr int kScalers = 4;                      // warps 4..7: a lane quarter each
    static constexpr int kReaders = 1 + kScalers + 1 + kPublishers;
    // tensor memory: two accumulators of gate and up (16 token columns each),
    // then for each stage the scales of four weight and four token tiles
    static constexpr int kTmemCols = 256, kSfCol = 64, kSfStage = 32;
};

template <int NT>
struct FewShared {   // after the ring
    uint64_t full[16], empty[16], sf_full[16];
    uint64_t unit_full[kUnitSlots], unit_empty[kUnitSlots];
    uint64_t res_full[2], res_empty[2], drain;
    uint32_t tmem_slot;
    int32_t unit[kUnitSlots];
    int abort, n_groups;
    int32_t ids[kMaxSlots];
    float wts[kMaxSlots];
    int16_t slot_row[kMaxSlots], first_id[kMaxSlots];
    int16_t group_id[kMaxGroups], group_row[kMaxGroups];
    uint8_t group_n[kMaxGroups], row_tok[kMaxRows];
    // a unit's 128 results of each token; the pitch keeps the stores conflict-free
    alignas(16) float res[2][8 * NT][132];
};

// Ring stages: what fits beside FewShared in the 227 KB a CTA can have.
template <int DT, int NT>
struct Ring {
    static constexpr int kAlign = DT == DT_MX4 ? 1024 : 128;
    static constexpr int kStages =
        (227 * 1024 - kAlign - (int)sizeof(FewShared<NT>)) / Traits<DT, NT>::kStage;
    static constexpr int kBytes = kAlign + kStages * Traits<DT, NT>::kStage + (int)sizeof(FewShared<NT>);
};
static_assert(Ring<DT_FP8, 1>::kStages == 5 && Ring<DT_FP8, 2>::kStages == 5 &&
              Ring<DT_MX4, 1>::kStages == 5 && Ring<DT_MX4, 2>::kStages == 5, "depth of the rings");

// Order-preserving integers of the selection values: larger is better, 0 is
// not selectable (NaN and minus infinity, as warp_select treats them); the two
// zeros are equal.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v >= -FLT_MAX)) return 0u;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return k == 0u ? -FLT_MAX : __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}

// Zeroes the keys of the groups that are not kept.  Lane g scores group g: the
// sum of its best, best first.
__device__ __forceinline__ void drop_groups(const SelectArgs &a, int lane, uint32_t *key) {
    const int gs = a.E / a.groups;
    float sum = 0.0f;
    if (lane < a.groups) {
        const uint32_t *k0 = key + lane * gs;
        if (a.topn <= 2) {   // the two largest values in one pass
            uint32_t m1 = 0, m2 = 0;
            int e = lane % gs;   // lanes start apart: one bank each where gs is a multiple of 32
#pragma unroll 4
            for (int i = 0; i < gs; ++i) {
                const uint32_t k = k0[e];
                m2 = max(m2, min(m1, k));
                m1 = max(m1, k);
                if (++e == gs) e = 0;
            }
            sum = key_value(m1);
            if (a.topn == 2) sum = __fadd_rn(sum, key_value(m2));
        } else {
            uint32_t pk = 0xffffffffu;
            int pi = -1;
            for (int r = 0; r < a.topn; ++r) {   // the next one in (value, index) order
                uint32_t bk = 0;
                int bi = INT_MAX;
                for (int e = 0; e < gs; ++e) {
                    const uint32_t k = k0[e];
                    if ((k < pk || (k == pk && e > pi)) && k > bk) bk = k, bi = e;
                }
                sum = r == 0 ? key_value(bk) : __fadd_rn(sum, key_value(bk));
                pk = bk;
                pi = bi;
            }
        }
    }
    const uint32_t gk = lane < a.groups ? order_key(sum) : 0u;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
        const uint32_t o = __shfl_sync(0xffffffffu, gk, g);
        rank += o > gk || (o == gk && g < lane);
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, gk != 0u && rank < a.topk_groups);
    __syncwarp();
    for (int g = 0; g < a.groups; ++g)
        if (!((kept >> g) & 1u))
            for (int e = lane; e < gs; e += 32) key[g * gs + e] = 0u;
    __syncwarp();
}

// The top_k of a token in order, lane j keeping the j-th's index; false if
// there are fewer candidates.
__device__ __forceinline__ bool choose(const SelectArgs &a, int lane, const uint32_t *key, int &my_id) {
    if (a.E <= 256) {   // experts e = 32 q + lane in registers
        uint32_t k[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) k[q] = 32 * q + lane < a.E ? key[32 * q + lane] : 0u;
#pragma unroll 1
        for (int j = 0; j < a.k; ++j) {
            uint32_t best = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) best = max(best, k[q]);
            const uint32_t m = __reduce_max_sync(0xffffffffu, best);
            if (m == 0u) return false;
            int at = INT_MAX;
#pragma unroll
            for (int q = 7; q >= 0; --q)
                if (k[q] == m) at = 32 * q + lane;
            const int id = (int)__reduce_min_sync(0xffffffffu, (uint32_t)at);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (32 * q + lane == id) k[q] = 0u;
            if (lane == j) my_id = id;
        }
        return true;
    }
    uint32_t pk = 0xffffffffu;
    int pi = -1;
    for (int j = 0; j < a.k; ++j) {   // the next one in (value, index) order
        uint32_t bk = 0;
        int bi = INT_MAX;
        for (int e = lane; e < a.E; e += 32) {
            const uint32_t k = key[e];
            if ((k < pk || (k == pk && e > pi)) && k > bk) bk = k, bi = e;
        }
        pk = __reduce_max_sync(0xffffffffu, bk);
        if (pk == 0u) return false;
        pi = (int)__reduce_min_sync(0xffffffffu, (uint32_t)(bk == pk ? bi : INT_MAX));
        if (lane == j) my_id = pi;
    }
    return true;
}

// warp_select's choice and weights (the same bits).  Every CTA runs this once,
// with a cold instruction cache, so its length counts more than its work:
// warp_select's unrolled shuffles took 15 us of the 84 that one token of the
// 256-expert layer took, this takes 3.5.  key, score: this warp's rows of E
// in shared memory; ids, wts: the token's top_k.
__device__ __noinline__ void few_select(const SelectArgs &a, int lane, uint32_t *key, const float *score,
                                        int32_t *ids, float *wts) {
    if (a.groups > 1) drop_groups(a, lane, key);
    int my_id = 0;
    if (!choose(a, lane, key, my_id)) {
        if (lane == 0 && a.status) atomicOr(a.status, MOE_DEV_BAD_EXPERT_ID);   // fewer candidates than k
        return;
    }
    const float mine = score[my_id];
    float w = 0.0f;
    if (a.sigmoid) {
        float total = 0.0f;
        for (int j = 0; j < a.k; ++j) total = __fadd_rn(total, __shfl_sync(0xffffffffu, mine, j));
        w = a.norm ? __fmul_rn(__fdiv_rn(mine, total), a.scaling) : __fmul_rn(mine, a.scaling);
    } else {
        float m = -FLT_MAX;
        for (int e = lane; e < a.E; e += 32) m = fmaxf(m, score[e]);
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        auto ex = [&](float lv) -> double {   // as warp_select's
            const float d = __fsub_rn(lv, m);
            const float bb = __fsub_rn(d, lv);
            const float e = __fadd_rn(__fsub_rn(lv, __fsub_rn(d, bb)), __fsub_rn(-m, bb));
            const double x = (double)expf(d);
            return fma(x, (double)e, x);
        };
        const double mex = ex(mine);
        double denom = 0.0;
        if (a.norm) {
            for (int j = 0; j < a.k; ++j) denom += __shfl_sync(0xffffffffu, mex, j);
        } else {
            for (int e = lane; e < a.E; e += 32) denom += ex(score[e]);
            for (int o = 16; o >= 1; o >>= 1) denom += __shfl_xor_sync(0xffffffffu, denom, o);
        }
        w = (float)(mex / denom * (double)a.scaling);
    }
    if (lane < a.k) {
        int id = my_id;
        if (a.log2phys) {
            id = a.log2phys[my_id];
            if (id < 0 || id >= a.E) {
                if (a.status) atomicOr(a.status, MOE_DEV_BAD_EXPERT_ID);
                id = -1;
            }
        }
        ids[lane] = id;
        wts[lane] = w;
    }
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// two e4m3 codes (a half word) as fp16 values, exact
__device__ __forceinline__ void e4m3_half4(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=&r"(lo), "=&r"(hi)
        : "r"(codes));
}

// What a lane holds of the token side for one tile of K: the words of column
// g of each n-tile, and (FP8) the scales of columns 2t and 2t+1.
// Columns past the group's rows hold what the stage held before; their
// results are not used.
template <int DT, int NT>
struct TokenSide {
    uint32_t b[NT][Traits<DT, NT>::kBWords];
    float s[NT][2];   // FP8
};

template <int DT, int NT>
__device__ __forceinline__ void load_tokens(TokenSide<DT, NT> &f, const uint8_t *rows, int g, int t) {
    using TR = Traits<DT, NT>;
    auto put = [](uint32_t *d, const uint8_t *p) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
    };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const uint8_t *p = rows + (8 * n + g) * TR::kPitch;
        if (DT == DT_FP8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                put(&f.b[n][8 * h], p + (t + 4 * h) * 32);
                put(&f.b[n][8 * h + 4], p + (t + 4 * h) * 32 + 16);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) put(&f.b[n][4 * h], p + (t + 4 * h) * 16);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (DT == DT_FP8)
                f.s[n][i] = *reinterpret_cast<const float *>(rows + (8 * n + 2 * t + i) * TR::kPitch + 256);
        }
    }
}

// acc += (16 weight rows of a tile in shared memory) x (the token side).
// ra: this lane's first row of the tile (the second is ra + 8); ws: the
// tile's scale (FP8).
template <int DT, int NT>
__device__ __forceinline__ void tile_product(float (&acc)[NT][4], const uint8_t *tile, int ra, int t,
                                             const TokenSide<DT, NT> &f, float ws, bool second) {
    using TR = Traits<DT, NT>;
    float part[NT][4] = {};
    const int sw = ra & 7;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint8_t *p = tile + ra * 128 + (((t + 4 * h) ^ sw) << 4);
        const uint4 va = *reinterpret_cast<const uint4 *>(p);
        const uint4 vb = *reinterpret_cast<const uint4 *>(p + 8 * 128);
        const uint32_t a[4] = {va.x, va.y, va.z, va.w}, b[4] = {vb.x, vb.y, vb.z, vb.w};
        if (DT == DT_BF16) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (!n || second)
                        mma_bf16(part[n], a[2 * i], b[2 * i], a[2 * i + 1], b[2 * i + 1],
                                 f.b[n][4 * h + 2 * i], f.b[n][4 * h + 2 * i + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t a0, a2, b0, b2;
                e4m3_half4(a[j], a0, a2);
                e4m3_half4(b[j], b0, b2);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (!n || second)
                        mma_f16(part[n], a0, b0, a2, b2, f.b[n][(8 * h + 2 * j) % TR::kBWords],
                                f.b[n][(8 * h + 2 * j + 1) % TR::kBWords]);
            }
        }
    }
    // A tile's sums join the unit's outside the tensor cores, whose additions
    // cut off instead of rounding: over 448 steps of K that had grown to 2.5e-5.
    if (DT == DT_BF16) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] += part[n][i];
    } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float s0 = __fmul_rn(f.s[n][0], ws), s1 = __fmul_rn(f.s[n][1], ws);
            acc[n][0] = fmaf(part[n][0], s0, acc[n][0]);
            acc[n][1] = fmaf(part[n][1], s1, acc[n][1]);
            acc[n][2] = fmaf(part[n][2], s0, acc[n][2]);
            acc[n][3] = fmaf(part[n][3], s1, acc[n][3]);
        }
    }
}

// MXFP4: 128 weight rows x 64 of K against 16 token rows, scale bytes sf and
// sf + 1 (mx4_gemm.cu has the same product for many rows).
__host__ __device__ constexpr uint32_t few_idesc_mxf4(int sf) {
    return ((uint32_t)sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(16 >> 3) << 17) | (1u << 23) |
           ((uint32_t)(128 >> 4) << 24) | ((uint32_t)sf << 29);
}
__device__ __forceinline__ void mma_tile_mxf4(uint32_t d, uint32_t weights, uint32_t tokens, uint32_t sfw,
                                              uint32_t sft, bool accumulate) {
    const uint64_t wd = ptx::sdesc_k_sw64(weights), td = ptx::sdesc_k_sw64(tokens);
    ptx::mma_mxf4(d, wd, td, few_idesc_mxf4(0), sfw, sft, accumulate);
    ptx::mma_mxf4(d, wd + 2, td + 2, few_idesc_mxf4(2), sfw, sft, 1);
}

template <int DT, int NT>
__global__ void __launch_bounds__(kFfnThreads, 1)
    few_ffn_kernel(const FewArgs a, const SelectArgs sel, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ CUtensorMap tmH) {
    using TR = Traits<DT, NT>;
    constexpr bool MX4 = DT == DT_MX4;
    constexpr int kStages = Ring<DT, NT>::kStages;
    extern __shared__ uint8_t dsmem[];
    uint8_t *ring = dsmem + (-ptx::smem_u32(dsmem) & (Ring<DT, NT>::kAlign - 1));
    FewShared<NT> &sh = *reinterpret_cast<FewShared<NT> *>(ring + kStages * TR::kStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.full[s]), 2);   // the weights' thread, the tokens' warp
            ptx::mbar_init(ptx::smem_u32(&sh.empty[s]), TR::kMultipliers);
            if constexpr (MX4) ptx::mbar_init(ptx::smem_u32(&sh.sf_full[s]), TR::kScalers);
        }
        for (int s = 0; s < kUnitSlots; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.unit_full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.unit_empty[s]), TR::kReaders);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.res_full[s]), TR::kMultipliers);
            ptx::mbar_init(ptx::smem_u32(&sh.res_empty[s]), kPublishers);
        }
        ptx::mbar_init(ptx::smem_u32(&sh.drain), 1);
        ptx::fence_mbar_init();
        sh.abort = 0;
        sh.n_groups = 0;
    }
    if constexpr (MX4) {
        if (warp == 0) {
            ptx::tmem_alloc(ptx::smem_u32(&sh.tmem_slot), TR::kTmemCols);
            ptx::tmem_relinquish();
        }
        if (warp == kTokens && lane == 0) {
            ptx::tma_prefetch_desc(&tmX);
            ptx::tma_prefetch_desc(&tmH);
        }
        ptx::tc_fence_before();   // the address is read after the barriers below
    }
    ptx::pdl_launch_dependents();
    const int slots = a.T * a.k;
    if (sel.groups > 1 && warp == 1) {
        // A selection of made-up keys while the kernel before this one ends, so
        // that the real one finds its code in the instruction cache (one token of
        // the 256-expert layer: 73.4 -> 71.5 us, 87 -> 81 after an idle GPU).
        // Without groups the code is short, and this was 2 us slower after an
        // idle GPU (the 16-expert layer).
        uint32_t *keys = reinterpret_cast<uint32_t *>(ring);
        float *scores = reinterpret_cast<float *>(ring) + a.E;
        SelectArgs s = sel;
        s.log2phys = nullptr;
        s.status = nullptr;
        for (int e = lane; e < a.E; e += 32) keys[e] = 0x80000000u + e, scores[e] = 1.0f;
        __syncwarp();
        few_select(s, lane, keys, scores, sh.ids, sh.wts);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += kFfnThreads) sh.ids[i] = -1;
    ptx::pdl_wait();   // scores, quantised x, counters
    __syncthreads();

    // The shared experts' weights are needed whatever the selection says: to L2
    // while it runs and HBM is idle (a hint; each CTA its part of each block).
    if (warp == kWarps - 1)
        for (int p = 0; p < 2; ++p) {
            const size_t bytes = p ? a.pf_w2 : a.pf_w13;   // of all shared experts, at most kPrefetchMost
            const uint8_t *w = p ? a.w2 + a.E * a.pf_w2_one : a.w13 + a.E * a.pf_w13_one;
            for (size_t o = ((size_t)lane * gridDim.x + blockIdx.x) * kPrefetchBytes; o < bytes;
                 o += (size_t)32 * gridDim.x * kPrefetchBytes)
                ptx::prefetch_l2(w + o, (uint32_t)min((size_t)kPrefetchBytes, bytes - o));
        }

    // ---- selection, by every CTA for itself -------------------------------------
    int next = 0;
    if (warp == kProducer && lane == 0) next = atomicAdd(a.sched, 1);   // the first unit
    {   // keys and scores of a token where the ring will be
        uint32_t *keys = reinterpret_cast<uint32_t *>(ring);
        float *scores = reinterpret_cast<float *>(ring) + a.T * a.E;
        for (int t = warp; t < a.T; t += kWarps) {
            uint32_t *key = keys + t * a.E;
            float *score = scores + t * a.E;
#pragma unroll 4
            for (int e = lane; e < a.E; e += 32) {
                key[e] = order_key(a.select[(size_t)t * a.E + e]);
                score[e] = a.score[(size_t)t * a.E + e];
            }
            __syncwarp();
            few_select(sel, lane, key, score, sh.ids + t * a.k, sh.wts + t * a.k);
        }
    }
    ptx::fence_proxy_async_shared();   // copies write there from here on
    __syncthreads();

    // ---- groups with rows: shared experts, then the chosen ones by id ----------
    // rows: shared expert s of token t at s T + t, then each chosen expert's
    // tokens in order.  A group takes 8 NT of them: a table log2phys with an
    // entry twice can give an expert more rows than there are tokens, which
    // are then further groups of the same weights.
    for (int i = threadIdx.x; i < slots; i += kFfnThreads) {
        const int id = sh.ids[i];
        int before = 0, rank = 0;   // slots of lower experts; of this one in earlier slots
        for (int j = 0; j < slots; ++j) {
            const int o = sh.ids[j];
            before += o >= 0 && o < id;
            rank += o == id && j < i;
        }
        const int row = id >= 0 ? a.S * a.T + before + rank : -1;
        if (id >= 0) sh.row_tok[row] = i / a.k;
        sh.slot_row[i] = row;
        sh.first_id[i] = id >= 0 && rank % (8 * NT) == 0 ? id : INT16_MAX;   // opens a group
        if (blockIdx.x == 0) {
            a.ids[i] = id;
            a.wts[i] = id >= 0 ? sh.wts[i] : 0.0f;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += kFfnThreads) {
        const int id = sh.first_id[i];
        if (id == INT16_MAX) continue;
        int place = a.S, n = 0;   // groups of lower experts, or before in this one; rows from here on
        for (int j = 0; j < slots; ++j) {
            place += sh.first_id[j] < id || (sh.first_id[j] == id && j < i);
            n += sh.ids[j] == id && j >= i;
        }
        sh.group_id[place] = id;
        sh.group_row[place] = sh.slot_row[i];
        sh.group_n[place] = min(n, 8 * NT);
        atomicAdd(&sh.n_groups, 1);
    }
    for (int i = threadIdx.x; i < a.S * a.T; i += kFfnThreads) sh.row_tok[i] = i % a.T;
    if (threadIdx.x < a.S) {
        sh.group_id[threadIdx.x] = a.E + threadIdx.x;
        sh.group_row[threadIdx.x] = threadIdx.x * a.T;
        sh.group_n[threadIdx.x] = a.T;
    }
    __syncthreads();

    uint32_t tmem = 0;
    if constexpr (MX4) {
        ptx::tc_fence_after();
        tmem = sh.tmem_slot;
    }
    const int nG = sh.n_groups + a.S;
    const int mt1 = a.I / 128, nb2 = a.H / 128;                  // tiles of 128 weight rows
    const int kb1 = a.H / TR::kKT, kb2 = a.I / TR::kKT;          // tiles along K
    const int u1 = nG * mt1, units = u1 + nG * nb2;              // no groups: no units
    int32_t *h_done = a.sched + 1, *col_done = h_done + kMaxGroups;
    volatile int *abort_flag = &sh.abort;

    if (nG == 0) {   // no shared expert and no valid choice: zeros
        const size_t n = (size_t)a.T * a.H;
        for (size_t i = (size_t)blockIdx.x * kFfnThreads + threadIdx.x; i < n;
             i += (size_t)gridDim.x * kFfnThreads) {
            if (a.out_bf16) static_cast<uint16_t *>(a.out)[i] = 0;
            else static_cast<float *>(a.out)[i] = 0.0f;
        }
    }

    // What a unit number stands for.
    struct Unit {
        bool gu;
        int gi, tile, kb, steps, per;   // a stage takes `per` tiles along K (gate/up: of both blocks)
    };
    auto unit_of = [&](int u) {
        Unit r;
        r.gu = u < u1;
        const int v = r.gu ? u : u - u1, per = r.gu ? mt1 : nb2;
        r.gi = v / per;
        r.tile = v % per;
        r.kb = r.gu ? kb1 : kb2;
        r.per = r.gu ? TR::kTiles / 2 : TR::kTiles;
        r.steps = (r.kb + r.per - 1) / r.per;
        return r;
    };
    // The it-th unit of this CTA (-1: no more), as every warp but the producer
    // reads it; -2 after a wait that gave up.
    auto take_unit = [&](int it) {
        const int slot = it % kUnitSlots;
        const bool ok = ptx::wait_bounded(ptx::smem_u32(&sh.unit_full[slot]), (it / kUnitSlots) & 1,
                                          abort_flag, a.status, MOE_DEV_TIMEOUT);
        if (!__all_sync(0xffffffffu, ok)) return -2;
        const int u = *reinterpret_cast<volatile int32_t *>(&sh.unit[slot]);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.unit_empty[slot]));
        return u;
    };

    if (warp == kProducer && lane == 0) {
        // ---- weights -------------------------------------------------------------
        const uint64_t policy = ptx::policy_evict_first();
        int issued = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int u = next, slot = it % kUnitSlots;
            if (!ptx::wait_bounded(ptx::smem_u32(&sh.unit_empty[slot]), ((it / kUnitSlots) & 1) ^ 1,
                                   abort_flag, a.status, MOE_DEV_TIMEOUT))
                break;
            sh.unit[slot] = u < units ? u : -1;
            ptx::mbar_arrive(ptx::smem_u32(&sh.unit_full[slot]));
            if (u >= units) break;
            const Unit un = unit_of(u);
            const size_t g = sh.group_id[un.gi];
            // tiles of a block of 128 weight rows are consecutive along K
            const size_t b0 = un.gu ? (g * 2 * mt1 + un.tile) * un.kb : (g * nb2 + un.tile) * un.kb;
            const size_t b1 = b0 + (size_t)mt1 * un.kb;   // the matching up rows
            const uint8_t *w = un.gu ? a.w13 : a.w2;
            const uint8_t *ws = static_cast<const uint8_t *>(un.gu ? a.w13_s : a.w2_s);
            for (int s = 0; s < un.steps; ++s) {
                const int st = issued % kStages;
                const uint32_t full = ptx::smem_u32(&sh.full[st]);
                if (!ptx::wait_bounded(ptx::smem_u32(&sh.empty[st]), ((issued / kStages) & 1) ^ 1,
                                       abort_flag, a.status, MOE_DEV_TIMEOUT)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = ptx::smem_u32(ring + st * TR::kStage);
                // `nk` tiles of a row block are consecutive: one copy
                const int k0 = s * un.per, nk = min(un.per, un.kb - k0);
                ptx::mbar_arrive_expect_tx(full, (un.gu ? 2 : 1) * nk * (TR::kTile + TR::kScale));
                for (int h = 0; h < (un.gu ? 2 : 1); ++h) {   // up in the second half of the stage
                    const size_t i = (h ? b1 : b0) + k0;
                    const uint32_t at = h * (TR::kTiles / 2);
                    ptx::bulk_load(dst + at * TR::kTile, w + i * TR::kTile, nk * TR::kTile, full, policy);
                    if constexpr (MX4)
                        ptx::bulk_load(dst + TR::kScaleOff + at * TR::kScale, ws + i * TR::kScale, nk * TR::kScale,
                                       full, policy);
                }
                ++issued;
            }
            // claimed only now: a unit claimed ahead would wait behind this one
            // while another CTA is idle.  The ring covers the counter's latency.
            next = atomicAdd(a.sched, 1);
        }
        // no copy may still be writing when the CTA's shared memory is given up
        for (int i = max(0, issued - kStages); i < issued; ++i)
            ptx::wait_drain(ptx::smem_u32(&sh.full[i % kStages]), (i / kStages) & 1);
    } else if (warp == kTokens) {
        // ---- the token side: x, or h once it is complete ------------------------------
        const uint64_t policy = ptx::policy_evict_last();
        ptx::fence_proxy_async_global();   // x's segments were written by another kernel
        int stage = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int u = take_unit(it);
            if (u < 0) break;
            const Unit un = unit_of(u);
            const int g = sh.group_id[un.gi], row0 = sh.group_row[un.gi], n = sh.group_n[un.gi];
            // FP8: the weight scales of the unit's row blocks, K tile i in lane i mod 32
            float wsc[2][2] = {};
            if (DT == DT_FP8) {
                const float *s0 = static_cast<const float *>(un.gu ? a.w13_s : a.w2_s) +
                                  (un.gu ? ((size_t)g * 2 * mt1 + un.tile) * un.kb
                                         : ((size_t)g * nb2 + un.tile) * un.kb);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (lane + 32 * i < un.kb) {
                        wsc[0][i] = __ldg(s0 + lane + 32 * i);
                        if (un.gu) wsc[1][i] = __ldg(s0 + (size_t)mt1 * un.kb + lane + 32 * i);
                    }
            }
            if (!un.gu) {   // all units of the group's h, from whichever CTAs
                ok = lane ? true
                          : ptx::wait_flag_geq(h_done + un.gi, mt1 * kPublishers, abort_flag, a.status, MOE_DEV_TIMEOUT);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                __syncwarp();   // what lane 0 has acquired, for every lane (the vote orders no memory)
                ptx::fence_proxy_async_global();
            }
            // this lane copies row `lane` (its segment of each K tile is contiguous)
            const int r = lane % (8 * NT), half = lane / (8 * NT);
            const uint8_t *src = nullptr;
            if (r < n && half < 2)
                src = un.gu ? a.xrows + (size_t)sh.row_tok[row0 + r] * un.kb * TR::kCopyX
                            : a.hrows + (size_t)(row0 + r) * un.kb * TR::kCopyH;
            const uint32_t copy = un.gu ? TR::kCopyX : TR::kCopyH;
            for (int s = 0; s < un.steps; ++s, ++stage) {
                const int st = stage % kStages;
                const uint32_t full = ptx::smem_u32(&sh.full[st]);
                ok = ptx::wait_bounded(ptx::smem_u32(&sh.empty[st]), ((stage / kStages) & 1) ^ 1, abort_flag,
                                       a.status, MOE_DEV_TIMEOUT);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint8_t *base = ring + st * TR::kStage;
                const int k0 = s * un.per, nk = min(un.per, un.kb - k0);
                if constexpr (MX4) {
                    // 16 rows whatever the group's: x's are all tokens, h's
                    // begin at the group's first (rows past its last are not used)
                    if (lane == 0) {
                        const uint32_t dst = ptx::smem_u32(base);
                        ptx::mbar_arrive_expect_tx(full, nk * (TR::kTokBytes + TR::kTokScale));
                        for (int k = 0; k < nk; ++k) {
                            ptx::tma_load_2d(dst + TR::kTokOff + k * TR::kTokBytes, un.gu ? &tmX : &tmH,
                                             (k0 + k) * 64, un.gu ? 0 : row0, full, policy);
                            const uint8_t *ts = un.gu ? a.xs + (size_t)(k0 + k) * kMaxT * kScaleRow
                                                      : a.hs + ((size_t)(k0 + k) * a.hs_rows + row0) * kScaleRow;
                            ptx::bulk_load(dst + TR::kTokScaleOff + k * 512, ts, TR::kTokScale, full, policy);
                        }
                    }
                    continue;
                }
                if (DT == DT_FP8) {
                    const int k1 = un.gu ? k0 : min(k0 + 1, un.kb - 1);
                    const float w0 = __shfl_sync(0xffffffffu, k0 < 32 ? wsc[0][0] : wsc[0][1], k0 & 31);
                    const float o0 = __shfl_sync(0xffffffffu, k1 < 32 ? wsc[0][0] : wsc[0][1], k1 & 31);
                    const float o1 = __shfl_sync(0xffffffffu, k1 < 32 ? wsc[1][0] : wsc[1][1], k1 & 31);
                    if (lane == 0)
                        *reinterpret_cast<float2 *>(base + TR::kWsOff) = make_float2(w0, un.gu ? o1 : o0);
                }
                if (lane == 0) ptx::mbar_arrive_expect_tx(full, n * nk * copy);
                __syncwarp();   // the bytes are announced before any copy lands
                if (src && half < nk)
                    ptx::bulk_load(ptx::smem_u32(base + TR::kTokOff + half * TR::kTokHalf + r * TR::kPitch),
                                   src + (size_t)(k0 + half) * copy, copy, full, policy);
            }
        }
        if (lane == 0)   // as the producer: no copy may outlive the CTA
            for (int i = max(0, stage - kStages); i < stage; ++i)
                ptx::wait_drain(ptx::smem_u32(&sh.full[i % kStages]), (i / kStages) & 1);
    } else if (warp >= kFirstPublisher) {
        // ---- results: h to its format and to memory, y to memory, the combine --------
        const int pw = warp - kFirstPublisher;
        // Each of the four warps finishes a unit for itself: no barrier among
        // them.  In a down unit warp quarter `q` has 32 of the 128 columns.
        const int q = MX4 ? warp & 3 : pw;   // MXFP4: the lane quarter the warp can read
        // Combines columns [32 q, 32 q + 32) of a tile for all tokens: lane
        // i = (token, four columns).
        auto combine = [&](int tile) {
            for (int i = lane; i < a.T * 8; i += 32) {
                const int t = i >> 3;
                const size_t col = tile * 128 + 32 * q + (i & 7) * 4;
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f), sr[kMaxShared], r[8];
                const float *y = a.y + col;
                auto load = [&](int j0) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int row = j0 + j < a.k ? sh.slot_row[t * a.k + j0 + j] : -1;
                        if (row >= 0) r[j] = __ldcg(reinterpret_cast<const float4 *>(y + (size_t)row * a.H));
                    }
                };
#pragma unroll
                for (int s = 0; s < kMaxShared; ++s)   // all loads first, then the sums in order
                    if (s < a.S)
                        sr[s] = __ldcg(reinterpret_cast<const float4 *>(y + (size_t)(s * a.T + t) * a.H));
                load(0);
#pragma unroll
                for (int s = 0; s < kMaxShared; ++s)
                    if (s < a.S) {
                        o.x = __fadd_rn(o.x, sr[s].x), o.y = __fadd_rn(o.y, sr[s].y);
                        o.z = __fadd_rn(o.z, sr[s].z), o.w = __fadd_rn(o.w, sr[s].w);
                    }
                for (int j0 = 0; j0 < a.k; j0 += 8) {
                    if (j0) load(j0);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (j0 + j >= a.k || sh.slot_row[t * a.k + j0 + j] < 0) continue;
                        const float w = sh.wts[t * a.k + j0 + j];
                        o.x = fmaf(w, r[j].x, o.x), o.y = fmaf(w, r[j].y, o.y);
                        o.z = fmaf(w, r[j].z, o.z), o.w = fmaf(w, r[j].w, o.w);
                    }
                }
                const size_t at = (size_t)t * a.H + col;
                if (a.out_bf16) {
                    __nv_bfloat162 b0 = __floats2bfloat162_rn(o.x, o.y), b1 = __floats2bfloat162_rn(o.z, o.w);
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
                        make_uint2(*reinterpret_cast<uint32_t *>(&b0), *reinterpret_cast<uint32_t *>(&b1));
                } else {
                    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = o;
                }
            }
        };
        // A down unit's count comes back while the next unit is worked on.
        int pending = -1, before = 0;
        auto finish_pending = [&]() {
            if (pending >= 0 && __shfl_sync(0xffffffffu, before, 0) == nG - 1) {
                // all groups' rows of these columns are there: for lane 0 by its
                // fence after the count, for the others by the barrier (the
                // shuffle orders no memory)
                __threadfence();
                __syncwarp();
                combine(pending);
            }
            pending = -1;
        };
        for (int it = 0;; ++it) {
            const int u = take_unit(it);
            if (u < 0) break;
            const Unit un = unit_of(u);
            const int row0 = sh.group_row[un.gi], n = sh.group_n[un.gi], buf = it & 1;
            const bool ok = ptx::wait_bounded(ptx::smem_u32(&sh.res_full[buf]), (it >> 1) & 1, abort_flag,
                                              a.status, MOE_DEV_TIMEOUT);
            if (!__all_sync(0xffffffffu, ok)) break;
            if constexpr (MX4) {
                // this warp's lane quarter of tensor memory: 32 of the 128 rows,
                // for gate/up one block of h's scales
                const int m = 32 * q + lane;
                const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + buf * 32;
                uint32_t d[16], up[16];
                ptx::tc_fence_after();
                ptx::tmem_ld16(acc, d);
                if (un.gu) ptx::tmem_ld16(acc + 16, up);
                ptx::tmem_wait_ld(d);
                ptx::tmem_wait_ld(up);
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.res_empty[buf]));
                if (un.gu) {
#pragma unroll
                    for (int c = 0; c < 8 * NT; ++c)
                        sh.res[0][c][m] = silu_mul(__uint_as_float(d[c]), __uint_as_float(up[c]));
                    __syncwarp();
                    for (int i0 = 0; i0 < n; i0 += 8) {   // eight rows, four lanes each
                        const int i = i0 + (lane >> 2), ch = lane & 3;
                        const size_t row = row0 + min(i, n - 1);
                        const float *p = &sh.res[0][sh.row_tok[row]][32 * q + 8 * ch];
                        float f[8];
                        *reinterpret_cast<float4 *>(f) = *reinterpret_cast<const float4 *>(p);
                        *reinterpret_cast<float4 *>(f + 4) = *reinterpret_cast<const float4 *>(p + 4);
                        uint32_t mx = 0;
#pragma unroll
                        for (int j = 0; j < 8; ++j) mx = max(mx, __float_as_uint(f[j]) & 0x7fffffffu);
                        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        const uint32_t byte = mx4_scale_byte(mx);
                        if (i < n) {
                            *reinterpret_cast<uint32_t *>(a.hrows + (row * a.I + un.tile * 128 + 32 * q + 8 * ch) / 2) =
                                mx4_codes8(f, byte);
                            if (ch == 0)
                                a.hs[((size_t)un.tile * a.hs_rows + row) * kScaleRow + q] = (uint8_t)byte;
                        }
                    }
                    __syncwarp();   // res is rewritten by the next unit
                } else {
#pragma unroll
                    for (int c = 0; c < 8 * NT; ++c)
                        if (c < n) a.y[(size_t)(row0 + c) * a.H + un.tile * 128 + m] = __uint_as_float(d[c]);
                }
            }
            if constexpr (!MX4) {
                if (un.gu) {
                    for (int c = pw; c < n; c += kPublishers) {
                        const float4 v = *reinterpret_cast<const float4 *>(&sh.res[buf][c][lane * 4]);
                        const size_t row = row0 + c;
                        if (DT == DT_BF16) {
                            const __nv_bfloat162 b0 = __floats2bfloat162_rn(v.x, v.y),
                                                 b1 = __floats2bfloat162_rn(v.z, v.w);
                            const float2 f0 = __bfloat1622float2(b0), f1 = __bfloat1622float2(b1);
                            // nothing is left of an infinity (inf - inf would add a NaN)
                            auto left = [](float all, float hi) { return fabsf(hi) <= FLT_MAX ? all - hi : 0.0f; };
                            const __nv_bfloat162 l0 = __floats2bfloat162_rn(left(v.x, f0.x), left(v.y, f0.y)),
                                                 l1 = __floats2bfloat162_rn(left(v.z, f1.x), left(v.w, f1.y));
                            // tile of 64: un.tile * 2 + lane / 16
                            uint8_t *o = a.hrows + ((row * mt1 + un.tile) * 2 + lane / 16) * TR::kCopyH + lane % 16 * 8;
                            auto bits = [](const __nv_bfloat162 &b) { return *reinterpret_cast<const uint32_t *>(&b); };
                            *reinterpret_cast<uint2 *>(o) = make_uint2(bits(b0), bits(b1));
                            *reinterpret_cast<uint2 *>(o + 128) = make_uint2(bits(l0), bits(l1));
                        } else {
                            uint8_t *seg = a.hrows + (row * mt1 + un.tile) * kSegment;
                            float m = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
                            for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                            const float sc = fp8_group_scale(m), inv = fp8_group_inv(sc);
                            const uint2 o = fp8_as_half4(__fmul_rn(v.x, inv), __fmul_rn(v.y, inv),
                                                         __fmul_rn(v.z, inv), __fmul_rn(v.w, inv));
                            if (lane == 0) *reinterpret_cast<float *>(seg + 256) = sc;
                            *reinterpret_cast<uint2 *>(seg + lane * 8) = o;
                        }
                    }
                } else {
                    for (int c = 0; c < n; ++c)
                        a.y[(size_t)(row0 + c) * a.H + un.tile * 128 + 32 * q + lane] = sh.res[buf][c][32 * q + lane];
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.res_empty[buf]));
            }
            if (un.gu) ptx::fence_proxy_async_global();   // h is read by copies
            __syncwarp();
            finish_pending();
            // the warp's stores, then (one fence by one lane, after the warp's
            // barrier) the count
            if (un.gu) {
                if (lane == 0) ptx::red_release_gpu_add(h_done + un.gi, 1);
            } else {
                if (lane == 0) {
                    __threadfence();
                    before = atomicAdd(col_done + un.tile * kPublishers + q, 1);
                }
                pending = un.tile;
            }
        }
        finish_pending();
    } else if constexpr (MX4) {
        // ---- products (MXFP4): one thread issues them -------------------------------
        if (warp == 0) {
            int stage = 0;
            bool ok = true;
            for (int it = 0; ok; ++it) {
                const int u = take_unit(it);
                if (u < 0) break;
                const Unit un = unit_of(u);
                const int buf = it & 1;
                if (lane == 0) {
                    ok = ptx::wait_bounded(ptx::smem_u32(&sh.res_empty[buf]), ((it >> 1) & 1) ^ 1, abort_flag,
                                           a.status, MOE_DEV_TIMEOUT);
                    ptx::tc_fence_after();
                    const uint32_t acc = tmem + buf * 32;
                    for (int s = 0; ok && s < un.steps; ++s) {
                        const int st = (stage + s) % kStages;
                        ok = ptx::wait_bounded(ptx::smem_u32(&sh.sf_full[st]), ((stage + s) / kStages) & 1,
                                               abort_flag, a.status, MOE_DEV_TIMEOUT);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint32_t base = ptx::smem_u32(ring + st * TR::kStage);
                        const uint32_t sf = tmem + TR::kSfCol + st * TR::kSfStage;
                        const int nk = min(un.per, un.kb - s * un.per);
                        for (int k = 0; k < nk; ++k) {
                            const uint32_t tok = base + TR::kTokOff + k * TR::kTokBytes;
                            mma_tile_mxf4(acc, base + k * TR::kTile, tok, sf + 4 * k, sf + 16 + 4 * k, s + k > 0);
                            if (un.gu)   // the up rows against the same tokens
                                mma_tile_mxf4(acc + 16, base + (k + 2) * TR::kTile, tok, sf + 4 * (k + 2),
                                              sf + 16 + 4 * k, s + k > 0);
                        }
                        ptx::mma_commit(ptx::smem_u32(&sh.empty[st]));
                    }
                    if (ok) ptx::mma_commit(ptx::smem_u32(&sh.res_full[buf]));
                }
                stage += un.steps;
                ok = __shfl_sync(0xffffffffu, (int)ok, 0);
            }
            if (lane == 0) {   // every product has landed before the columns are given up
                ptx::mma_commit(ptx::smem_u32(&sh.drain));
                ptx::wait_drain(ptx::smem_u32(&sh.drain), 0);
            }
        } else if (warp >= kConsumers - TR::kScalers && warp < kConsumers) {
            // ---- scales to tensor memory: each of these warps writes its lane
            // quarter.  The tensor pipe's own copies (tcgen05.cp) took about 100
            // cycles each in line with products of about 118, three to every four.
            const uint32_t quarter = (uint32_t)(warp & 3) << 21;   // lane 32 (warp & 3)
            int stage = 0;
            bool ok = true;
            for (int it = 0; ok; ++it) {
                const int u = take_unit(it);
                if (u < 0) break;
                const Unit un = unit_of(u);
                for (int s = 0; s < un.steps; ++s, ++stage) {
                    const int st = stage % kStages;
                    ok = ptx::wait_bounded(ptx::smem_u32(&sh.full[st]), (stage / kStages) & 1, abort_flag,
                                           a.status, MOE_DEV_TIMEOUT);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    ptx::tc_fence_after();   // the products that read these columns before are done
                    const uint8_t *base = ring + st * TR::kStage;
                    const uint32_t sf = tmem + quarter + TR::kSfCol + st * TR::kSfStage;
                    const int nk = min(un.per, un.kb - s * un.per);
#pragma unroll
                    for (int k = 0; k < TR::kTiles; ++k)   // a slot without a tile: not used
                        ptx::tmem_st4(sf + 4 * k, *reinterpret_cast<const uint4 *>(
                                                      base + TR::kScaleOff + k * TR::kScale + lane * 16));
                    for (int k = 0; k < nk; ++k)
                        ptx::tmem_st1(sf + 16 + 4 * k, *reinterpret_cast<const uint32_t *>(
                                                           base + TR::kTokScaleOff + k * 512 + lane * 16));
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.sf_full[st]));
                }
            }
        }
    } else if (warp < kConsumers) {
        // ---- products ---------------------------------------------------------------
        const int g8 = lane >> 2, t4 = lane & 3;
        const int ra = warp * 16 + ((g8 >> 1) | ((g8 & 1) << 2));   // this lane's rows ra, ra + 8
        int stage = 0;   // stages consumed so far
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int u = take_unit(it);
            if (u < 0) break;
            const Unit un = unit_of(u);
            const int n = sh.group_n[un.gi];
            const bool second = NT > 1 && n > 8;
            float acc[2][NT][4] = {};
            for (int s = 0; s < un.steps; ++s, ++stage) {
                const int st = stage % kStages;
                ok = ptx::wait_bounded(ptx::smem_u32(&sh.full[st]), (stage / kStages) & 1, abort_flag, a.status,
                                       MOE_DEV_TIMEOUT);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint8_t *base = ring + st * TR::kStage;
                float2 ws = make_float2(0.0f, 0.0f);
                if (DT == DT_FP8) ws = *reinterpret_cast<const float2 *>(base + TR::kWsOff);
                TokenSide<DT, NT> f;
                load_tokens<DT, NT>(f, base + TR::kTokOff, g8, t4);
                tile_product<DT, NT>(acc[0], base, ra, t4, f, ws.x, second);
                if (DT == DT_BF16 && !un.gu) {   // h's low part
                    load_tokens<DT, NT>(f, base + TR::kTokOff + 128, g8, t4);
                    tile_product<DT, NT>(acc[0], base, ra, t4, f, ws.x, second);
                }
                if (un.gu) {
                    tile_product<DT, NT>(acc[1], base + TR::kTile, ra, t4, f, ws.y, second);
                } else if (2 * s + 1 < un.kb) {
                    load_tokens<DT, NT>(f, base + TR::kTokOff + TR::kTokHalf, g8, t4);
                    tile_product<DT, NT>(acc[0], base + TR::kTile, ra, t4, f, ws.y, second);
                    if (DT == DT_BF16) {
                        load_tokens<DT, NT>(f, base + TR::kTokOff + TR::kTokHalf + 128, g8, t4);
                        tile_product<DT, NT>(acc[0], base + TR::kTile, ra, t4, f, ws.y, second);
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[st]));
            }
            if (!ok) break;
            const int buf = it & 1;
            ok = ptx::wait_bounded(ptx::smem_u32(&sh.res_empty[buf]), ((it >> 1) & 1) ^ 1, abort_flag, a.status,
                                   MOE_DEV_TIMEOUT);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = 8 * j + 2 * t4 + (i & 1);
                    if (c < n)
                        sh.res[buf][c][ra + (i & 2) * 4] =
                            un.gu ? silu_mul(acc[0][j][i], acc[1][j][i]) : acc[0][j][i];
                }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.res_full[buf]));
        }
    }

    if constexpr (MX4) {
        __syncwarp();
        ptx::tc_fence_before();
        __syncthreads();
        if (warp == 0) {
            ptx::tc_fence_after();
            ptx::tmem_dealloc(tmem, TR::kTmemCols);
        }
    }
}

template <int DT, int NT>
int launch_ffn(const FewArgs &a, const SelectArgs &sel, cudaStream_t s) {
    CUtensorMap tmX = {}, tmH = {};
    if (DT == DT_MX4) {
        const int rows = a.T * (a.k + a.S);
        if (!encode_2d_sw64(&tmX, a.xrows, (uint64_t)a.H / 2, (uint64_t)a.T, 16) ||
            !encode_2d_sw64(&tmH, a.hrows, (uint64_t)a.I / 2, (uint64_t)rows, 16))
            return cuda_fail("cuTensorMapEncodeTiled (token rows)");
    }
    constexpr int smem = Ring<DT, NT>::kBytes;
    static std::once_flag once[64];
    static int rc[64];
    int dev = 0;
    MOE_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return cuda_fail("device ordinal beyond 63");
    std::call_once(once[dev], [&] {
        rc[dev] = (int)cudaFuncSetAttribute(few_ffn_kernel<DT, NT>,
                                            cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (rc[dev]) return cuda_fail("cudaFuncSetAttribute", (cudaError_t)rc[dev]);
    return launch_dependent(few_ffn_kernel<DT, NT>, dim3(sm_count()), dim3(kFfnThreads), smem, s, a,
                            sel, tmX, tmH);
}

int sched_ints(const moe_config *c) { return 1 + kMaxGroups + c->hidden / 128 * kPublishers; }

}  // namespace

void few_layout(const moe_config *c, moe_few_layout *L) {
    const int64_t T = c->max_tokens, H = c->hidden, I = c->inter, k = c->top_k;
    const int64_t R = T * (k + c->num_shared);
    const bool bf = c->dtype == MOE_DTYPE_BF16, mx4 = c->dtype == MOE_DTYPE_MXFP4;
    size_t off = 0;
    auto take = [&](int64_t bytes) {
        const size_t o = off;
        off = align_up(off + (size_t)bytes);
        return o;
    };
    L->status = take(4);
    L->sched = take(4 * (int64_t)sched_ints(c));
    L->score = take(4 * T * c->num_experts);
    L->select = take(4 * T * c->num_experts);
    L->topk_ids = take(4 * T * k);
    L->topk_w = take(4 * T * k);
    L->x = take(bf ? 0 : mx4 ? T * H / 2 : T * (H / 128) * kSegment);
    L->x_scales = take(mx4 ? H / 128 * kMaxT * kScaleRow : 0);
    L->h = take(bf ? 4 * R * I : mx4 ? R * I / 2 : R * (I / 128) * kSegment);
    // a box of 16 rows may begin at any row
    L->h_scales = take(mx4 ? I / 128 * (R + kMaxT) * kScaleRow : 0);
    L->y = take(4 * R * H);
    L->total = off;
}

int launch_layer_few(const moe_config *c, const moe_weights *w, int T, const void *x, void *out,
                     int out_dtype, void *ws, cudaStream_t s) {
    moe_few_layout L;
    few_layout(c, &L);
    uint8_t *b = static_cast<uint8_t *>(ws);
    const int H = c->hidden, E = c->num_experts, S = c->num_shared;

    SelectArgs sel = {};
    sel.T = T;
    sel.E = E;
    sel.k = c->top_k;
    sel.groups = c->num_groups;
    sel.topk_groups = c->topk_groups;
    sel.topn = c->group_topn;
    sel.sigmoid = c->scoring == MOE_SCORING_SIGMOID;
    sel.norm = c->norm_topk;
    sel.scaling = c->routed_scaling;
    sel.bias = w->e_bias;
    sel.log2phys = w->log2phys;
    sel.status = reinterpret_cast<int32_t *>(b + L.status);

    RouteArgs r = {};
    r.T = T;
    r.H = H;
    r.E = E;
    r.sched_ints = sched_ints(c);
    r.dtype = c->dtype;
    r.x = static_cast<const uint16_t *>(x);
    r.wg = static_cast<const uint16_t *>(w->w_gate);
    r.offset = w->logit_offset;
    r.sel = sel;
    r.score = reinterpret_cast<float *>(b + L.score);
    r.select = reinterpret_cast<float *>(b + L.select);
    r.xq = b + L.x;
    r.xs = b + L.x_scales;
    r.sched = reinterpret_cast<int32_t *>(b + L.sched);
    r.status = sel.status;
    const int64_t warps = (int64_t)E * ceil_div(T, kTokChunk);
    r.logit_blocks = (int)ceil_div(warps, kRouteThreads / 32);
    const int64_t qwarps = c->dtype == MOE_DTYPE_BF16 ? 0 : (int64_t)T * ceil_div(H, 256);
    const int64_t blocks = r.logit_blocks + ceil_div(qwarps, kRouteThreads / 32);
    if (int rc = launch_dependent(few_route_kernel, dim3((unsigned)blocks), dim3(kRouteThreads), 0, s, r))
        return rc;

    FewArgs a = {};
    a.T = T;
    a.H = H;
    a.I = c->inter;
    a.E = E;
    a.S = S;
    a.k = c->top_k;
    a.out_bf16 = out_dtype == MOE_OUT_BF16;
    a.w13 = static_cast<const uint8_t *>(w->w13);
    a.w2 = static_cast<const uint8_t *>(w->w2);
    a.w13_s = w->w13_scales;
    a.w2_s = w->w2_scales;
    const size_t IH = (size_t)c->inter * H;   // elements of W2
    a.pf_w2_one = c->dtype == MOE_DTYPE_MXFP4 ? IH / 2 : c->dtype == MOE_DTYPE_BF16 ? 2 * IH : IH;
    a.pf_w13_one = 2 * a.pf_w2_one;
    a.pf_w13 = std::min(S * a.pf_w13_one, kPrefetchMost);
    a.pf_w2 = std::min(S * a.pf_w2_one, kPrefetchMost);
    a.score = r.score;
    a.select = r.select;
    a.ids = reinterpret_cast<int32_t *>(b + L.topk_ids);
    a.wts = reinterpret_cast<float *>(b + L.topk_w);
    a.xrows = c->dtype == MOE_DTYPE_BF16 ? static_cast<const uint8_t *>(x) : r.xq;
    a.hrows = b + L.h;
    a.xs = r.xs;
    a.hs = b + L.h_scales;
    a.hs_rows = c->max_tokens * (c->top_k + S) + kMaxT;
    a.y = reinterpret_cast<float *>(b + L.y);
    a.out = out;
    a.sched = r.sched;
    a.status = r.status;
    switch (c->dtype) {
    case MOE_DTYPE_BF16: return T <= 8 ? launch_ffn<DT_BF16, 1>(a, sel, s) : launch_ffn<DT_BF16, 2>(a, sel, s);
    case MOE_DTYPE_FP8_BLOCK128: return T <= 8 ? launch_ffn<DT_FP8, 1>(a, sel, s) : launch_ffn<DT_FP8, 2>(a, sel, s);
    default: return T <= 8 ? launch_ffn<DT_MX4, 1>(a, sel, s) : launch_ffn<DT_MX4, 2>(a, sel, s);
    }
}

}  // namespace moe
