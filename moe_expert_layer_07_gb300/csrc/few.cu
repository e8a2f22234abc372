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
// at the copy rate, for one token of nine 44 MB experts.  Everything else has
// to hide behind that stream: a producer thread keeps a ring of weight tiles
// (MOE_LAYOUT_TILES, one bulk copy each) full, and runs ahead into the next
// unit, and into the down products, while the consumers still wait for h.
//
// Units, claimed in order from a counter: for every active group (an expert
// with rows) and 128 of its features, gate and up (2 x 128 weight rows against
// the group's token rows; h = silu(g) u, rounded or quantised, to global
// memory); then for every active group and 128 hidden columns, down.  A down
// unit waits (bounded) until its group's h is complete.  Every unit that is
// waited for was claimed before by a running CTA, which finishes it without
// waiting for anyone, so no co-residency is assumed.  The CTA that adds the
// last group's rows to a block of 128 columns combines them for all tokens, in
// the combine kernel's order: no atomic sums, the result does not depend on
// who came when.
//
// The products use the warp-wide MMA (m16n8): 16 weight rows of a warp on its
// M side, up to 8 tokens on N.  tcgen05 would leave its 128-row tile's
// accumulators to be read back and scaled per 128 of K in FP8; here they are
// already in registers, and the tensor rate does not matter: at 24 bytes of
// weights a clock and SM the warps' MMA is under a quarter busy.  A thread
// reads 16 bytes of a weight row at a time (the order of K inside a product is
// free as long as both sides agree), rows 0, 4, 1, 5, ... of eight in MMA
// order, which makes the reads conflict-free on the swizzled tiles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "internal.h"
#include "mx4.cuh"
#include "numerics.cuh"
#include "ptx.cuh"
#include "route_select.cuh"

namespace moe {
namespace {

constexpr int kMaxT = kFewMaxTokens;
constexpr int kMaxShared = 4;
constexpr int kMaxSlots = kMaxT * 16;                   // routed slots
constexpr int kMaxRows = kMaxSlots + kMaxT * kMaxShared;
constexpr int kMaxGroups = kMaxSlots + kMaxShared;      // groups with rows

enum { DT_BF16 = MOE_DTYPE_BF16, DT_FP8 = MOE_DTYPE_FP8_BLOCK128, DT_MX4 = MOE_DTYPE_MXFP4 };

struct FewArgs {
    int T, H, I, E, S, k, out_bf16;
    const uint16_t *x;          // bf16 [T, H]
    const uint8_t *w13, *w2;
    const void *w13_s, *w2_s;
    const float *logits;
    int32_t *ids;
    float *wts;
    const uint16_t *x16;        // what the products read: bf16 x, or fp16 code values
    const void *xs;             // fp32 [T, H/128] (FP8) or scale bytes [T, H/32] (MXFP4)
    uint16_t *h16;
    void *hs;
    float *y;                   // [rows, H]
    void *out;
    int32_t *sched;             // unit counter | h_done[kMaxGroups] | col_done[H/128]
    int32_t *status;
};

// ---- kernel 1 ---------------------------------------------------------------

constexpr int kRouteThreads = 128;
constexpr int kTokChunk = 4;   // tokens a warp takes against one gate row

struct RouteArgs {
    int T, H, E, sched_ints, logit_blocks, dtype;
    const uint16_t *x, *wg;
    const float *offset;
    float *logits;
    uint16_t *x16;
    void *xs;
    int32_t *sched, *status;
    const uint8_t *pf[2];       // weights to bring into L2 (the shared experts')
    size_t pf_bytes[2];
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
    constexpr int U = NT == 1 ? 14 : 7;   // loads in flight
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
// (quant_row_segment's arithmetic, or mx4.cu's), each code kept as the fp16
// number it stands for before its scale.
__device__ __forceinline__ void quant_segment(const RouteArgs &a, int t, int seg, int lane) {
    const int col = seg * 256 + lane * 8;
    const bool active = col < a.H;
    float f[8] = {};
    if (active) bf8(__ldg(reinterpret_cast<const uint4 *>(a.x + (size_t)t * a.H + col)), f);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
    uint4 o;
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
        o = make_uint4(p.x, p.y, q.x, q.y);
        if (active && (lane & 15) == 0)
            static_cast<float *>(a.xs)[(size_t)t * (a.H / 128) + col / 128] = sc;
    } else {
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t byte = mx4_scale_byte(m);
        uint32_t h[4];
        mx4_half8(mx4_codes8(f, byte), h);
        o = make_uint4(h[0], h[1], h[2], h[3]);
        if (active && (lane & 3) == 0)
            static_cast<uint8_t *>(a.xs)[(size_t)t * (a.H / 32) + col / 32] = (uint8_t)byte;
    }
    if (active) *reinterpret_cast<uint4 *>(a.x16 + (size_t)t * a.H + col) = o;
}

__global__ void __launch_bounds__(kRouteThreads) few_route_kernel(const RouteArgs a) {
    ptx::pdl_launch_dependents();
    const int gtid = blockIdx.x * kRouteThreads + threadIdx.x, nthreads = gridDim.x * kRouteThreads;
#pragma unroll
    for (int p = 0; p < 2; ++p)   // a hint: 16 KB for each thread that takes part
        for (size_t o = (size_t)gtid * 16384; o < a.pf_bytes[p]; o += (size_t)nthreads * 16384)
            ptx::prefetch_l2(a.pf[p] + o, (uint32_t)min((size_t)16384, a.pf_bytes[p] - o));
    ptx::pdl_wait();   // x, and the last call's use of the workspace
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    for (int i = gtid; i < a.sched_ints; i += nthreads) a.sched[i] = 0;
    const int warp = (blockIdx.x * kRouteThreads + threadIdx.x) >> 5;
    if ((int)blockIdx.x >= a.logit_blocks) {
        const int q = warp - a.logit_blocks * (kRouteThreads / 32), segs = (a.H + 255) / 256;
        if (q < a.T * segs) quant_segment(a, q / segs, q % segs, lane);
        return;
    }
    const int chunks = (a.T + kTokChunk - 1) / kTokChunk;
    const int e = warp / chunks, t0 = warp % chunks * kTokChunk;
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
        if (lane == t && t < nt)
            a.logits[(size_t)(t0 + t) * a.E + e] = a.offset ? __fadd_rn(v, a.offset[e]) : v;
    }
}

// ---- kernel 2 ---------------------------------------------------------------

constexpr int kConsumers = 8;                         // consumer warps
constexpr int kFfnThreads = (kConsumers + 1) * 32;    // and the producer's

template <int DT>
struct Traits {
    // K elements of one tile, bytes of its codes and of its scales in a stage
    static constexpr int kKT = DT == DT_BF16 ? 64 : 128;
    static constexpr int kTile = DT == DT_MX4 ? 8192 : 16384;
    static constexpr int kScale = DT == DT_MX4 ? 512 : 0;
    static constexpr int kStage = 2 * (kTile + kScale);
    static constexpr int kStages = DT == DT_MX4 ? 11 : 6;
    static constexpr int kBWords = DT == DT_BF16 ? 8 : 16;   // B words a lane holds for a tile
};

struct FewShared {   // after the ring
    uint64_t full[16], empty[16];
    uint64_t unit_full[2], unit_empty[2];
    uint64_t sync;
    int32_t unit[2];
    int abort, last, n_groups;
    int32_t ids[kMaxSlots], slot_row[kMaxSlots], first_id[kMaxSlots];
    float wts[kMaxSlots];
    int32_t group_id[kMaxGroups], group_row[kMaxGroups], group_n[kMaxGroups];
    int32_t row_tok[kMaxRows];
    alignas(16) float h[kMaxT][132];   // 128 features of a token; the pitch keeps the stores conflict-free
};

template <int PL>
__device__ __noinline__ void select_tokens(const SelectArgs &a, float *sh, int warp, int lane) {
    float *l = sh + warp * 3 * PL * 32, *s = l + PL * 32, *sel = s + PL * 32;
    for (int t = warp; t < a.T; t += kConsumers) {
        for (int e = lane; e < PL * 32; e += 32) {
            const bool ok = e < a.E;
            const float lv = ok ? a.logits[(size_t)t * a.E + e] : 0.0f;
            float sv, selv;
            expert_scores(a, e, ok, lv, sv, selv);
            l[e] = lv;
            s[e] = sv;
            sel[e] = selv;
        }
        __syncwarp();
        warp_select<PL>(a, t, lane, l, s, sel);
        __syncwarp();
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
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}

// What a lane holds of the token side for one tile of K: the words of column
// g of each n-tile, and (scaled types) the scales of columns 2t and 2t+1.
template <int DT, int NT>
struct TokenSide {
    uint32_t b[NT][Traits<DT>::kBWords];
    float s[NT][2];        // FP8
    uint32_t s4[NT][2];    // MXFP4: four scale bytes, one for each 32 of K
};

template <int DT, int NT, bool FRESH>   // FRESH: written during this kernel (past L1)
__device__ __forceinline__ void load_tokens(TokenSide<DT, NT> &f, const uint16_t *const (&row)[NT],
                                            const uint8_t *const (&srow)[NT][2], int kb, int t) {
    using TR = Traits<DT>;
    auto ld = [](const uint16_t *p) {
        return FRESH ? __ldcg(reinterpret_cast<const uint4 *>(p))
                     : *reinterpret_cast<const uint4 *>(p);
    };
    auto put = [](uint32_t *d, const uint4 v) { d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w; };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const uint16_t *p = row[n];
        if (p) {
            p += (size_t)kb * TR::kKT;
            if (DT == DT_FP8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    put(&f.b[n][8 * h], ld(p + (t + 4 * h) * 16));
                    put(&f.b[n][8 * h + 4], ld(p + (t + 4 * h) * 16 + 8));
                }
            } else if (DT == DT_BF16) {
#pragma unroll
                for (int h = 0; h < 2; ++h) put(&f.b[n][4 * h], ld(p + (t + 4 * h) * 8));
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) put(&f.b[n][4 * q], ld(p + q * 32 + t * 8));
            }
        } else {
#pragma unroll
            for (int i = 0; i < TR::kBWords; ++i) f.b[n][i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (DT == DT_FP8) {
                const float *q = reinterpret_cast<const float *>(srow[n][i]) + kb;
                f.s[n][i] = srow[n][i] ? (FRESH ? __ldcg(q) : *q) : 0.0f;
            } else if (DT == DT_MX4) {
                const uint32_t *q = reinterpret_cast<const uint32_t *>(srow[n][i]) + kb;
                f.s4[n][i] = srow[n][i] ? (FRESH ? __ldcg(q) : *q) : 0x7f7f7f7fu;
            }
        }
    }
}

// acc += (16 weight rows of a tile in shared memory) x (the token side).
// ra: this lane's first row of the tile (the second is ra + 8); ws: the
// tile's scale (FP8); scales: its scale bytes in shared memory (MXFP4).
template <int DT, int NT>
__device__ __forceinline__ void tile_product(float (&acc)[NT][4], const uint8_t *tile, int ra, int t,
                                             const TokenSide<DT, NT> &f, float ws, bool second) {
    if (DT == DT_MX4) {
        const uint8_t *scales = tile + Traits<DT>::kTile;
        const uint32_t sa4 = *reinterpret_cast<const uint32_t *>(scales + (ra & 31) * 16 + (ra >> 5) * 4);
        const int rb = ra + 8;
        const uint32_t sb4 = *reinterpret_cast<const uint32_t *>(scales + (rb & 31) * 16 + (rb >> 5) * 4);
        const int sw = (ra >> 1) & 3;   // the swizzle of both rows
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint8_t *p = tile + ra * 64 + ((q ^ sw) << 4) + t * 4;
            uint32_t a[4], b[4];
            mx4_half8(*reinterpret_cast<const uint32_t *>(p), a);
            mx4_half8(*reinterpret_cast<const uint32_t *>(p + 8 * 64), b);
            const float wa = mx4_scale((sa4 >> (8 * q)) & 255u), wb = mx4_scale((sb4 >> (8 * q)) & 255u);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n && !second) continue;
                float part[4] = {};
                mma_f16(part, a[0], b[0], a[1], b[1], f.b[n][4 * q], f.b[n][4 * q + 1]);
                mma_f16(part, a[2], b[2], a[3], b[3], f.b[n][4 * q + 2], f.b[n][4 * q + 3]);
                const float x0 = mx4_scale((f.s4[n][0] >> (8 * q)) & 255u);
                const float x1 = mx4_scale((f.s4[n][1] >> (8 * q)) & 255u);
                acc[n][0] = fmaf(part[0] * wa, x0, acc[n][0]);
                acc[n][1] = fmaf(part[1] * wa, x1, acc[n][1]);
                acc[n][2] = fmaf(part[2] * wb, x0, acc[n][2]);
                acc[n][3] = fmaf(part[3] * wb, x1, acc[n][3]);
            }
        }
        return;
    }
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
                        mma_bf16(acc[n], a[2 * i], b[2 * i], a[2 * i + 1], b[2 * i + 1],
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
                        mma_f16(part[n], a0, b0, a2, b2, f.b[n][8 * h + 2 * j],
                                f.b[n][8 * h + 2 * j + 1]);
            }
        }
    }
    if (DT == DT_FP8) {
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

template <int DT, int NT>
__global__ void __launch_bounds__(kFfnThreads, 1)
    few_ffn_kernel(const FewArgs a, const SelectArgs sel) {
    using TR = Traits<DT>;
    extern __shared__ __align__(1024) uint8_t ring[];
    FewShared &sh = *reinterpret_cast<FewShared *>(ring + TR::kStages * TR::kStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < TR::kStages; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.empty[s]), kConsumers);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.unit_full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.unit_empty[s]), kConsumers);
        }
        ptx::mbar_init(ptx::smem_u32(&sh.sync), kConsumers);
        ptx::fence_mbar_init();
        sh.abort = 0;
        sh.n_groups = 0;
    }
    const int slots = a.T * a.k;
    for (int i = threadIdx.x; i < slots; i += kFfnThreads) sh.ids[i] = -1;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();   // logits, quantised x, counters
    __syncthreads();

    // ---- selection, by every CTA for itself (scores where the ring will be) ----
    if (warp < kConsumers) {
        SelectArgs s = sel;
        s.ids = sh.ids;
        s.w = sh.wts;
        float *buf = reinterpret_cast<float *>(ring);
        if (s.E <= 32) select_tokens<1>(s, buf, warp, lane);
        else if (s.E <= 64) select_tokens<2>(s, buf, warp, lane);
        else if (s.E <= 128) select_tokens<4>(s, buf, warp, lane);
        else if (s.E <= 256) select_tokens<8>(s, buf, warp, lane);
        else if (s.E <= 512) select_tokens<16>(s, buf, warp, lane);
        else select_tokens<32>(s, buf, warp, lane);
    }
    __syncthreads();

    // ---- groups with rows: shared experts, then the chosen ones by id ----------
    // rows: shared expert s of token t at s T + t, then each chosen expert's
    // tokens in order
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
        sh.first_id[i] = id >= 0 && rank == 0 ? id : INT_MAX;
        if (blockIdx.x == 0) {
            a.ids[i] = id;
            a.wts[i] = id >= 0 ? sh.wts[i] : 0.0f;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += kFfnThreads) {
        const int id = sh.first_id[i];
        if (id == INT_MAX) continue;
        int place = a.S, n = 0;   // distinct chosen experts below; this one's rows
        for (int j = 0; j < slots; ++j) {
            place += sh.first_id[j] < id;
            n += sh.ids[j] == id;
        }
        sh.group_id[place] = id;
        sh.group_row[place] = sh.slot_row[i];
        sh.group_n[place] = n;
        atomicAdd(&sh.n_groups, 1);
    }
    for (int i = threadIdx.x; i < a.S * a.T; i += kFfnThreads) sh.row_tok[i] = i % a.T;
    if (threadIdx.x < a.S) {
        sh.group_id[threadIdx.x] = a.E + threadIdx.x;
        sh.group_row[threadIdx.x] = threadIdx.x * a.T;
        sh.group_n[threadIdx.x] = a.T;
    }
    ptx::fence_proxy_async_shared();   // the scores' place is written by copies from here on
    __syncthreads();

    const int nG = sh.n_groups + a.S;
    const int mt1 = a.I / 128, nb2 = a.H / 128;                  // tiles of 128 weight rows
    const int kb1 = a.H / TR::kKT, kb2 = a.I / TR::kKT;          // tiles along K
    const int u1 = nG * mt1, units = u1 + nG * nb2;
    int32_t *h_done = a.sched + 1, *col_done = h_done + kMaxGroups;
    volatile int *abort_flag = &sh.abort;

    if (nG == 0) {   // no shared expert and no valid choice: zeros
        const size_t n = (size_t)a.T * a.H;
        for (size_t i = (size_t)blockIdx.x * kFfnThreads + threadIdx.x; i < n;
             i += (size_t)gridDim.x * kFfnThreads) {
            if (a.out_bf16) static_cast<uint16_t *>(a.out)[i] = 0;
            else static_cast<float *>(a.out)[i] = 0.0f;
        }
        return;
    }

    if (warp == kConsumers) {
        // ---- producer ------------------------------------------------------------
        if (lane) return;
        const uint64_t policy = ptx::policy_evict_first();
        int issued = 0;
        bool ok = true;
        int next = atomicAdd(a.sched, 1);
        for (int it = 0; ok; ++it) {
            const int u = next;
            const int slot = it & 1;
            if (!ptx::wait_bounded(ptx::smem_u32(&sh.unit_empty[slot]), ((it >> 1) & 1) ^ 1,
                                   abort_flag, a.status, MOE_DEV_TIMEOUT))
                break;
            sh.unit[slot] = u < units ? u : -1;
            ptx::mbar_arrive(ptx::smem_u32(&sh.unit_full[slot]));
            if (u >= units) break;
            next = atomicAdd(a.sched, 1);
            const bool gu = u < u1;
            const int v = gu ? u : u - u1, per = gu ? mt1 : nb2;
            const int gi = v / per, tile = v % per, kb = gu ? kb1 : kb2;
            const size_t g = sh.group_id[gi];
            // tiles of a block of 128 weight rows are consecutive along K
            const size_t b0 = gu ? (g * 2 * mt1 + tile) * kb : (g * nb2 + tile) * kb;
            const size_t b1 = b0 + (size_t)mt1 * kb;   // the matching up rows
            const uint8_t *w = gu ? a.w13 : a.w2;
            const uint8_t *ws = static_cast<const uint8_t *>(gu ? a.w13_s : a.w2_s);
            const int steps = gu ? kb : (kb + 1) / 2;
            for (int s = 0; s < steps; ++s) {
                const int st = issued % TR::kStages;
                const uint32_t full = ptx::smem_u32(&sh.full[st]);
                if (!ptx::wait_bounded(ptx::smem_u32(&sh.empty[st]), ((issued / TR::kStages) & 1) ^ 1,
                                       abort_flag, a.status, MOE_DEV_TIMEOUT)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = ptx::smem_u32(ring + st * TR::kStage);
                constexpr uint32_t kSlot = TR::kTile + TR::kScale;
                const size_t i0 = gu ? b0 + s : b0 + 2 * s, i1 = gu ? b1 + s : i0 + 1;
                const bool two = gu || 2 * s + 1 < kb;
                ptx::mbar_arrive_expect_tx(full, two ? 2 * kSlot : kSlot);
                ptx::bulk_load(dst, w + i0 * TR::kTile, TR::kTile, full, policy);
                if (TR::kScale) ptx::bulk_load(dst + TR::kTile, ws + i0 * TR::kScale, TR::kScale, full, policy);
                if (two) {
                    ptx::bulk_load(dst + kSlot, w + i1 * TR::kTile, TR::kTile, full, policy);
                    if (TR::kScale)
                        ptx::bulk_load(dst + kSlot + TR::kTile, ws + i1 * TR::kScale, TR::kScale, full, policy);
                }
                ++issued;
            }
        }
        // no copy may still be writing when the CTA's shared memory is given up
        for (int i = max(0, issued - TR::kStages); i < issued; ++i)
            ptx::wait_drain(ptx::smem_u32(&sh.full[i % TR::kStages]), (i / TR::kStages) & 1);
        return;
    }

    // ---- consumers -----------------------------------------------------------------
    const int g8 = lane >> 2, t4 = lane & 3;
    const int ra = warp * 16 + ((g8 >> 1) | ((g8 & 1) << 2));   // this lane's rows ra, ra + 8
    uint32_t sync_parity = 0;
    auto consumer_sync = [&]() -> bool {   // all consumer warps; bounded
        __syncwarp();
        const uint32_t bar = ptx::smem_u32(&sh.sync);
        if (lane == 0) ptx::mbar_arrive(bar);
        const bool ok = ptx::wait_bounded(bar, sync_parity, abort_flag, a.status, MOE_DEV_TIMEOUT);
        sync_parity ^= 1;
        return __all_sync(0xffffffffu, ok);
    };
    int stage = 0;   // stages consumed so far
    bool ok = true;
    for (int it = 0; ok; ++it) {
        const int slot = it & 1;
        ok = ptx::wait_bounded(ptx::smem_u32(&sh.unit_full[slot]), (it >> 1) & 1, abort_flag, a.status,
                               MOE_DEV_TIMEOUT);
        if (!__all_sync(0xffffffffu, ok)) break;
        const int u = *reinterpret_cast<volatile int32_t *>(&sh.unit[slot]);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.unit_empty[slot]));
        if (u < 0) break;
        const bool gu = u < u1;
        const int v = gu ? u : u - u1, per = gu ? mt1 : nb2;
        const int gi = v / per, tile = v % per, kb = gu ? kb1 : kb2;
        const int g = sh.group_id[gi], row0 = sh.group_row[gi], n = sh.group_n[gi];
        const bool second = NT > 1 && n > 8;

        // the token side's rows: column 8 j + g8 of the MMA, scales of 2 t4 (+1)
        const uint16_t *rows[NT];
        const uint8_t *srows[NT][2];
        const uint16_t *src = gu ? a.x16 : a.h16;
        const uint8_t *ssrc = static_cast<const uint8_t *>(gu ? a.xs : a.hs);
        const int K = gu ? a.H : a.I, spitch = K / 32;   // bytes of scales a row, FP8 too
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            auto at = [&](int c) { return gu ? sh.row_tok[row0 + c] : row0 + c; };
            rows[j] = 8 * j + g8 < n ? src + (size_t)at(8 * j + g8) * K : nullptr;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = 8 * j + 2 * t4 + i;
                srows[j][i] = DT != DT_BF16 && c < n ? ssrc + (size_t)at(c) * spitch : nullptr;
            }
        }
        // FP8: the weight scales of the unit's row blocks, K block i in lane i mod 32
        float wsc[2][2] = {};
        if (DT == DT_FP8) {
            const float *s0 = static_cast<const float *>(gu ? a.w13_s : a.w2_s) +
                              (gu ? ((size_t)g * 2 * mt1 + tile) * kb : ((size_t)g * nb2 + tile) * kb);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (lane + 32 * i < kb) {
                    wsc[0][i] = __ldg(s0 + lane + 32 * i);
                    if (gu) wsc[1][i] = __ldg(s0 + (size_t)mt1 * kb + lane + 32 * i);
                }
        }
        if (!gu) {   // the group's h: all its units, from whichever CTAs
            ok = lane ? true
                      : ptx::wait_flag_geq(h_done + gi, mt1, abort_flag, a.status, MOE_DEV_TIMEOUT);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
        }
        float acc[2][NT][4] = {};
        TokenSide<DT, NT> cur, nxt;
        auto load = [&](TokenSide<DT, NT> &f, int i) {
            if (gu) load_tokens<DT, NT, false>(f, rows, srows, i, t4);
            else load_tokens<DT, NT, true>(f, rows, srows, i, t4);
        };
        load(cur, 0);
        for (int i = 0; i < kb; ++i) {
            if (i + 1 < kb) load(nxt, i + 1);
            const int st = stage % TR::kStages;
            const int half = gu ? 0 : i & 1;   // a down stage holds two K tiles
            if (half == 0) {
                ok = ptx::wait_bounded(ptx::smem_u32(&sh.full[st]), (stage / TR::kStages) & 1, abort_flag,
                                       a.status, MOE_DEV_TIMEOUT);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
            }
            constexpr int kSlot = TR::kTile + TR::kScale;
            const uint8_t *base = ring + st * TR::kStage;
            float w0 = 0.0f, w1 = 0.0f;
            if (DT == DT_FP8) {
                w0 = __shfl_sync(0xffffffffu, i < 32 ? wsc[0][0] : wsc[0][1], i & 31);
                w1 = __shfl_sync(0xffffffffu, i < 32 ? wsc[1][0] : wsc[1][1], i & 31);
            }
            tile_product<DT, NT>(acc[0], base + half * kSlot, ra, t4, cur, w0, second);
            if (gu) tile_product<DT, NT>(acc[1], base + kSlot, ra, t4, cur, w1, second);
            if (gu || half == 1 || i + 1 == kb) {
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[st]));
                ++stage;
            }
            cur = nxt;
        }
        if (!ok) break;

        if (gu) {
            // h = silu(gate) up: to shared memory, then quantised by token
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = 8 * j + 2 * t4 + (i & 1);
                    if (c < n) sh.h[c][ra + (i & 2) * 4] = silu_mul(acc[0][j][i], acc[1][j][i]);
                }
            if (!(ok = consumer_sync())) break;
            for (int c = warp; c < n; c += kConsumers) {
                const float4 q = *reinterpret_cast<const float4 *>(&sh.h[c][lane * 4]);
                uint2 o;
                const size_t row = row0 + c;
                if (DT == DT_BF16) {
                    __nv_bfloat162 b0 = __floats2bfloat162_rn(q.x, q.y), b1 = __floats2bfloat162_rn(q.z, q.w);
                    o = make_uint2(*reinterpret_cast<uint32_t *>(&b0), *reinterpret_cast<uint32_t *>(&b1));
                } else if (DT == DT_FP8) {
                    float m = fmaxf(fmaxf(fabsf(q.x), fabsf(q.y)), fmaxf(fabsf(q.z), fabsf(q.w)));
#pragma unroll
                    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                    const float sc = fp8_group_scale(m), inv = fp8_group_inv(sc);
                    o = fp8_as_half4(__fmul_rn(q.x, inv), __fmul_rn(q.y, inv), __fmul_rn(q.z, inv),
                                     __fmul_rn(q.w, inv));
                    if (lane == 0) static_cast<float *>(a.hs)[row * mt1 + tile] = sc;
                } else {
                    uint32_t m = max(max(__float_as_uint(q.x) & 0x7fffffffu, __float_as_uint(q.y) & 0x7fffffffu),
                                     max(__float_as_uint(q.z) & 0x7fffffffu, __float_as_uint(q.w) & 0x7fffffffu));
#pragma unroll
                    for (int d = 4; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
                    const uint32_t byte = mx4_scale_byte(m);
                    o = byte == 255u ? make_uint2(0u, 0u)
                                     : mx4_as_half4(q.x, q.y, q.z, q.w, mx4_inv_scale(byte));
                    if ((lane & 7) == 0)
                        static_cast<uint8_t *>(a.hs)[row * (a.I / 32) + tile * 4 + lane / 8] = (uint8_t)byte;
                }
                *reinterpret_cast<uint2 *>(a.h16 + row * a.I + tile * 128 + lane * 4) = o;
            }
            __threadfence();
            if (!(ok = consumer_sync())) break;   // every warp's rows are out; sh.h is free
            if (threadIdx.x == 0) ptx::red_release_gpu_add(h_done + gi, 1);
        } else {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = 8 * j + 2 * t4 + (i & 1);
                    if (c < n) a.y[(size_t)(row0 + c) * a.H + tile * 128 + ra + (i & 2) * 4] = acc[0][j][i];
                }
            __threadfence();
            if (!(ok = consumer_sync())) break;
            if (threadIdx.x == 0) {
                sh.last = atomicAdd(col_done + tile, 1) == nG - 1;
                __threadfence();
            }
            if (!(ok = consumer_sync())) break;
            if (!sh.last) continue;
            // all groups' rows of these columns are there: the combine
            for (int i = threadIdx.x; i < a.T * 32; i += kConsumers * 32) {
                const int t = i >> 5;
                const size_t col = tile * 128 + (i & 31) * 4;
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int s = 0; s < a.S; ++s) {
                    const float4 r = __ldcg(reinterpret_cast<const float4 *>(a.y + (size_t)(s * a.T + t) * a.H + col));
                    o.x = __fadd_rn(o.x, r.x), o.y = __fadd_rn(o.y, r.y);
                    o.z = __fadd_rn(o.z, r.z), o.w = __fadd_rn(o.w, r.w);
                }
                for (int j = 0; j < a.k; ++j) {
                    const int row = sh.slot_row[t * a.k + j];
                    if (row < 0) continue;
                    const float w = sh.wts[t * a.k + j];
                    const float4 r = __ldcg(reinterpret_cast<const float4 *>(a.y + (size_t)row * a.H + col));
                    o.x = fmaf(w, r.x, o.x), o.y = fmaf(w, r.y, o.y);
                    o.z = fmaf(w, r.z, o.z), o.w = fmaf(w, r.w, o.w);
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
        }
    }
}

template <int DT, int NT>
int launch_ffn(const FewArgs &a, const SelectArgs &sel, cudaStream_t s) {
    using TR = Traits<DT>;
    const int smem = TR::kStages * TR::kStage + (int)sizeof(FewShared);
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
                            sel);
}

int sched_ints(const moe_config *c) { return 1 + kMaxGroups + c->hidden / 128; }

}  // namespace

void few_layout(const moe_config *c, moe_few_layout *L) {
    const int64_t T = c->max_tokens, H = c->hidden, I = c->inter, k = c->top_k;
    const int64_t R = T * (k + c->num_shared);
    const bool bf = c->dtype == MOE_DTYPE_BF16, fp8 = c->dtype == MOE_DTYPE_FP8_BLOCK128;
    size_t off = 0;
    auto take = [&](int64_t bytes) {
        const size_t o = off;
        off = align_up(off + (size_t)bytes);
        return o;
    };
    L->status = take(4);
    L->sched = take(4 * (int64_t)sched_ints(c));
    L->logits = take(4 * T * c->num_experts);
    L->topk_ids = take(4 * T * k);
    L->topk_w = take(4 * T * k);
    L->x16 = take(bf ? 0 : 2 * T * H);
    L->xs = take(bf ? 0 : fp8 ? 4 * T * (H / 128) : T * (H / 32));
    L->h16 = take(2 * R * I);
    L->hs = take(bf ? 0 : fp8 ? 4 * R * (I / 128) : R * (I / 32));
    L->y = take(4 * R * H);
    L->total = off;
}

int launch_layer_few(const moe_config *c, const moe_weights *w, int T, const void *x, void *out,
                     int out_dtype, void *ws, cudaStream_t s) {
    moe_few_layout L;
    few_layout(c, &L);
    uint8_t *b = static_cast<uint8_t *>(ws);
    const int H = c->hidden, E = c->num_experts, S = c->num_shared;

    RouteArgs r = {};
    r.T = T;
    r.H = H;
    r.E = E;
    r.sched_ints = sched_ints(c);
    r.dtype = c->dtype;
    r.x = static_cast<const uint16_t *>(x);
    r.wg = static_cast<const uint16_t *>(w->w_gate);
    r.offset = w->logit_offset;
    r.logits = reinterpret_cast<float *>(b + L.logits);
    r.x16 = reinterpret_cast<uint16_t *>(b + L.x16);
    r.xs = b + L.xs;
    r.sched = reinterpret_cast<int32_t *>(b + L.sched);
    r.status = reinterpret_cast<int32_t *>(b + L.status);
    const int64_t warps = (int64_t)E * ceil_div(T, kTokChunk);
    r.logit_blocks = (int)ceil_div(warps, kRouteThreads / 32);
    const int64_t qwarps = c->dtype == MOE_DTYPE_BF16 ? 0 : (int64_t)T * ceil_div(H, 256);
    const int64_t blocks = r.logit_blocks + ceil_div(qwarps, kRouteThreads / 32);
    if (int rc = launch_dependent(few_route_kernel, dim3((unsigned)blocks), dim3(kRouteThreads), 0, s, r))
        return rc;

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
    sel.logits = r.logits;
    sel.bias = w->e_bias;
    sel.log2phys = w->log2phys;
    sel.status = r.status;

    FewArgs a = {};
    a.T = T;
    a.H = H;
    a.I = c->inter;
    a.E = E;
    a.S = S;
    a.k = c->top_k;
    a.out_bf16 = out_dtype == MOE_OUT_BF16;
    a.x = r.x;
    a.w13 = static_cast<const uint8_t *>(w->w13);
    a.w2 = static_cast<const uint8_t *>(w->w2);
    a.w13_s = w->w13_scales;
    a.w2_s = w->w2_scales;
    a.logits = r.logits;
    a.ids = reinterpret_cast<int32_t *>(b + L.topk_ids);
    a.wts = reinterpret_cast<float *>(b + L.topk_w);
    a.x16 = c->dtype == MOE_DTYPE_BF16 ? r.x : r.x16;
    a.xs = r.xs;
    a.h16 = reinterpret_cast<uint16_t *>(b + L.h16);
    a.hs = b + L.hs;
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
