// Grouped products of MXFP4 rows and weights:
//   C[r, n] = sum_k A[r, k] W[g, n, k]      (rows r of group g)
// on the tensor cores' block-scaled four-bit kind (tcgen05.mma kind::mxf4:
// e2m1 operands, one power-of-two scale for 32 of K, fp32 accumulation in
// tensor memory), with a plain epilogue (fp32 or bf16 C) or SwiGLU and the
// MXFP4 quantisation of h (gate block and up block of the same 128 features
// in one tile).
//
// One persistent CTA per SM takes tiles of 128 token rows (M) x 256 weight
// rows (N, two blocks of 128).  A stage of the ring holds 256 of K: the token
// rows' codes (TMA boxes of 64 bytes, 64-byte swizzle), four weight tiles (8
// KB bulk copies, stored pre-swizzled) with their scale bytes (512-byte bulk
// copies, stored in the order tensor memory wants), and the token rows' scale
// bytes, which come row-major from global memory and are put in that order by
// four warps, one for each ring slot: a warp's lane L holds rows L, L+32,
// L+64, L+96, whose four words of four scales are one 16-byte chunk.  The MMA
// thread copies scales to tensor memory (tcgen05.cp, 32 lanes x 16 bytes,
// repeated for the four lane quarters) in front of the products that use them.
//
// The hardware applies the scales, so nothing is promoted on the way and an
// accumulator runs over all of K; the epilogue sees each output once.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "internal.h"
#include "mx4.cuh"
#include "numerics.cuh"
#include "ptx.cuh"
#include "tma_host.h"

namespace moe {
namespace {

constexpr int kTM = 128, kTN = 256;
constexpr int kStages = 4;
constexpr int kTileBytes = 128 * 64;                     // 128 rows x 128 of K
constexpr int kAOff = 0, kBOff = 2 * kTileBytes;         // B: [K block][weight block]
constexpr int kSAOff = kBOff + 4 * kTileBytes;           // scales of the token rows, 512 each
constexpr int kSBOff = kSAOff + 2 * 512;                 // of the weights: [K block][weight block]
constexpr int kStageBytes = kSBOff + 4 * 512;
constexpr int kScaleWarps = 4, kEpiWarps = 8;
constexpr int kFirstScaleWarp = 2, kFirstEpiWarp = kFirstScaleWarp + kScaleWarps;
constexpr int kThreads = (kFirstEpiWarp + kEpiWarps) * 32;
constexpr int kMaxGroups = 1024;
constexpr int kSmemBytes = kStages * kStageBytes + 1024;
// tensor memory: the accumulator, then for each ring slot and K block the
// scales of the token rows (4 columns) and of the weight rows (8)
constexpr int kTmemCols = 512, kSfCol = kTN, kSfStage = 2 * (4 + 8);
static_assert(kScaleWarps == kStages, "scale warp i serves ring slot i");
static_assert(kSfCol + kStages * kSfStage <= kTmemCols, "tensor memory columns");
static_assert(kStageBytes % 1024 == 0, "stages keep the swizzle's alignment");

struct Mx4Args {
    int groups, n_out, k_dim, rows;
    const uint8_t *a_scales;   // [rows, k_dim / 32]
    const int32_t *offsets;
    const uint8_t *w, *w_scales;
    void *c;                   // plain: [rows, n_out]; SwiGLU: codes [rows, n_out / 4]
    uint8_t *h_scales;         // SwiGLU: [rows, n_out / 64]
    int c_bf16;
    int32_t *status;
};

// instruction descriptor: e2m1 x e2m1, ue8m0 scales, K = 64, scale bytes `sf`
// and `sf` + 1 of each 32-bit column
__host__ __device__ constexpr uint32_t idesc_mxf4(int sf) {
    return ((uint32_t)sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kTN >> 3) << 17) | (1u << 23) |
           ((uint32_t)(kTM >> 4) << 24) | ((uint32_t)sf << 29);
}

struct Tile {
    int g, nt, row0, nvalid;
};

// Tile t -> (group, column tile, first row, valid rows); s_tiles holds each
// group's first tile.  Row tiles of one column tile are neighbours, so they
// share its weights in L2.
__device__ __forceinline__ Tile decode(int t, int G, const int *s_tiles, const int *s_off) {
    int lo = 0, hi = G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tiles[mid] <= t) lo = mid;
        else hi = mid;
    }
    Tile w;
    w.g = lo;
    const int rows = s_off[lo + 1] - s_off[lo], mtiles = (rows + kTM - 1) / kTM;
    const int local = t - s_tiles[lo];
    w.nt = local / mtiles;
    const int mt = local - w.nt * mtiles;
    w.row0 = s_off[lo] + mt * kTM;
    w.nvalid = min(kTM, rows - mt * kTM);
    return w;
}

// 16 fp32 columns of a row to C
__device__ __forceinline__ void store16(const Mx4Args &a, size_t row, int col, const uint32_t (&r)[16]) {
    const size_t at = row * a.n_out + col;
    if (a.c_bf16) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            w[j] = *reinterpret_cast<uint32_t *>(&b);
        }
        uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.c) + at);
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
        uint4 *o = reinterpret_cast<uint4 *>(static_cast<float *>(a.c) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
    }
}

template <bool SW>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                    const Mx4Args args) {
    using namespace ptx;
    extern __shared__ uint8_t dsmem[];
    __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages], acc_full, acc_empty, drain_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_abort, s_bad;
    __shared__ int s_off[kMaxGroups + 1], s_tiles[kMaxGroups + 1];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t smem_base = (smem_u32(dsmem) + 1023u) & ~1023u;
    const int G = args.groups;
    const int nblocks = args.n_out / 128;                       // weight blocks of a group
    const int NT = SW ? nblocks / 2 : (nblocks + 1) / 2;        // column tiles
    const int KB = args.k_dim / 128, steps = (KB + 1) / 2;      // K blocks; ring stages a tile
    volatile int *abort_flag = &s_abort;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 2);   // the copies' thread and the scale warp
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
        mbar_init(smem_u32(&acc_full), 1);
        mbar_init(smem_u32(&acc_empty), kEpiWarps);
        mbar_init(smem_u32(&drain_bar), 1);
        s_abort = 0;
        s_bad = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmA32);
    }
    pdl_launch_dependents();
    pdl_wait();
    for (int i = threadIdx.x; i <= G; i += kThreads) s_off[i] = args.offsets[i];
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += kThreads) {
        const int a = s_off[g], b = s_off[g + 1];
        if (a < 0 || b < a || b > args.rows) s_bad = 1;
    }
    __syncthreads();
    auto tiles_of = [&](int g) { return NT * ((s_off[g + 1] - s_off[g] + kTM - 1) / kTM); };
    if (warp == 0 && !s_bad) {   // prefix over groups: lane L owns a contiguous run
        const int per = (G + 31) / 32, g0 = lane * per;
        int local = 0;
        for (int q = 0; q < per; ++q)
            if (g0 + q < G) local += tiles_of(g0 + q);
        int incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += n;
        }
        int run = incl - local;
        for (int q = 0; q < per; ++q)
            if (g0 + q < G) {
                s_tiles[g0 + q] = run;
                run += tiles_of(g0 + q);
            }
        if (lane == 31) s_tiles[G] = incl;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int total = s_bad ? 0 : s_tiles[G];
    if (s_bad && threadIdx.x == 0 && blockIdx.x == 0 && args.status)
        atomicOr(args.status, MOE_DEV_BAD_OFFSETS);

    if (warp == 0) {
        // ---- copies ---------------------------------------------------------------
        if (lane == 0) {
            const uint64_t pol_w = policy_evict_normal(), pol_a = policy_evict_last();
            uint32_t it = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const Tile tl = decode(t, G, s_tiles, s_off);
                const size_t b0 = (size_t)tl.g * nblocks + (SW ? tl.nt : 2 * tl.nt);
                const size_t b1 = SW ? b0 + NT : b0 + 1;
                const int nb = SW || 2 * tl.nt + 1 < nblocks ? 2 : 1;
                const bool wide = tl.nvalid > 96;   // one box of 128 rows, else boxes of 32
                const int boxes = wide ? 1 : (tl.nvalid + 31) / 32;
                const uint32_t abytes = (wide ? 128 : boxes * 32) * 64;
                for (int s = 0; s < steps; ++s, ++it) {
                    const uint32_t slot = it % kStages;
                    if (!wait_bounded(smem_u32(&empty_bar[slot]), ((it / kStages) & 1) ^ 1u, abort_flag,
                                      args.status, MOE_DEV_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    const uint32_t base = smem_base + slot * kStageBytes, fb = smem_u32(&full_bar[slot]);
                    const int nk = min(2, KB - 2 * s);
                    mbar_arrive_expect_tx(fb, nk * (abytes + nb * (kTileBytes + 512)));
                    for (int k = 0; k < nk; ++k) {
                        const int kb = 2 * s + k;
                        for (int q = 0; q < boxes; ++q)
                            tma_load_2d(base + kAOff + k * kTileBytes + q * 32 * 64, wide ? &tmA : &tmA32,
                                        kb * 64, tl.row0 + q * 32, fb, pol_a);
                        for (int n = 0; n < nb; ++n) {
                            const size_t tile = (n ? b1 : b0) * KB + kb;
                            bulk_load(base + kBOff + (2 * k + n) * kTileBytes, args.w + tile * kTileBytes,
                                      kTileBytes, fb, pol_w);
                            bulk_load(base + kSBOff + (2 * k + n) * 512, args.w_scales + tile * 512, 512, fb,
                                      pol_w);
                        }
                    }
                }
            }
            // copies in flight have to land before the CTA gives up its memory
            if (!ok)
                for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
                    wait_drain(smem_u32(&full_bar[i % kStages]), (i / kStages) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- products --------------------------------------------------------------
        if (lane == 0) {
            uint32_t it = 0, tiles = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x, ++tiles) {
                if (!wait_bounded(smem_u32(&acc_empty), (tiles & 1) ^ 1u, abort_flag, args.status,
                                  MOE_DEV_TIMEOUT))
                    break;
                tc_fence_after();
                for (int s = 0; s < steps; ++s, ++it) {
                    const uint32_t slot = it % kStages;
                    if (!wait_bounded(smem_u32(&full_bar[slot]), (it / kStages) & 1, abort_flag, args.status,
                                      MOE_DEV_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t base = smem_base + slot * kStageBytes;
                    const uint32_t sf = tmem + kSfCol + slot * kSfStage;
                    const int nk = min(2, KB - 2 * s);
                    for (int k = 0; k < nk; ++k) {
                        const uint32_t sfa = sf + k * 12, sfb = sfa + 4;
                        tmem_copy_scales(sfa, sdesc_scales(base + kSAOff + k * 512));
                        tmem_copy_scales(sfb, sdesc_scales(base + kSBOff + 2 * k * 512));
                        tmem_copy_scales(sfb + 4, sdesc_scales(base + kSBOff + (2 * k + 1) * 512));
                        const uint64_t ad = sdesc_k_sw64(base + kAOff + k * kTileBytes);
                        const uint64_t bd = sdesc_k_sw64(base + kBOff + 2 * k * kTileBytes);
                        mma_mxf4(tmem, ad, bd, idesc_mxf4(0), sfa, sfb, s + k > 0);
                        mma_mxf4(tmem, ad + 2, bd + 2, idesc_mxf4(2), sfa, sfb, 1);
                    }
                    mma_commit(smem_u32(&empty_bar[slot]));
                }
                if (ok) mma_commit(smem_u32(&acc_full));
            }
            mma_commit(smem_u32(&drain_bar));
            wait_drain(smem_u32(&drain_bar), 0);
        }
        __syncwarp();
    } else if (warp < kFirstEpiWarp) {
        // ---- scales of the token rows ------------------------------------------------
        const uint32_t mine = warp - kFirstScaleWarp;   // this warp's ring slot
        uint8_t *smem = dsmem + (smem_base - smem_u32(dsmem));
        const size_t pitch = args.k_dim / 32;
        uint32_t it = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Tile tl = decode(t, G, s_tiles, s_off);
            for (int s = 0; s < steps; ++s, ++it) {
                if (it % kStages != mine) continue;
                const int nk = min(2, KB - 2 * s);
                uint32_t v[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = lane + 32 * j;
                        v[k][j] = 0x7f7f7f7fu;
                        if (k < nk && r < tl.nvalid)
                            v[k][j] = __ldg(reinterpret_cast<const uint32_t *>(
                                args.a_scales + (size_t)(tl.row0 + r) * pitch + (2 * s + k) * 4));
                    }
                ok = wait_bounded(smem_u32(&empty_bar[mine]), ((it / kStages) & 1) ^ 1u, abort_flag,
                                  args.status, MOE_DEV_TIMEOUT);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    *reinterpret_cast<uint4 *>(smem + mine * kStageBytes + kSAOff + k * 512 + lane * 16) =
                        make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&full_bar[mine]));
            }
        }
    } else {
        // ---- epilogue ------------------------------------------------------------------
        const int q = warp & 3, half = (warp - kFirstEpiWarp) >> 2;   // lane quarter, column half
        const int m = 32 * q + lane;                                  // this thread's row of the tile
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16);
        uint32_t tiles = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x, ++tiles) {
            const Tile tl = decode(t, G, s_tiles, s_off);
            const bool ok = wait_bounded(smem_u32(&acc_full), tiles & 1, abort_flag, args.status,
                                         MOE_DEV_TIMEOUT);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const bool valid = m < tl.nvalid;
            const size_t row = tl.row0 + m;
            if (SW) {
                uint16_t sc = 0;
#pragma unroll
                for (int b = 0; b < 2; ++b) {   // 32 features, one block of scales
                    float h[32];
                    uint32_t amax = 0;
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        uint32_t g[16], u[16];
                        const uint32_t col = half * 64 + b * 32 + p * 16;
                        tmem_ld16(lane_base + col, g);
                        tmem_ld16(lane_base + 128 + col, u);
                        tmem_wait_ld(g);
                        tmem_wait_ld(u);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float v = silu_mul(__uint_as_float(g[j]), __uint_as_float(u[j]));
                            h[16 * p + j] = v;
                            amax = max(amax, __float_as_uint(v) & 0x7fffffffu);
                        }
                    }
                    const uint32_t byte = mx4_scale_byte(amax);
                    sc |= (uint16_t)(byte << (8 * b));
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = h[8 * j + i];
                        o[j] = mx4_codes8(v, byte);
                    }
                    if (valid)
                        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(args.c) + row * (args.n_out / 4) +
                                                   tl.nt * 64 + half * 32 + b * 16) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                }
                if (valid)
                    *reinterpret_cast<uint16_t *>(args.h_scales + row * (args.n_out / 64) + tl.nt * 4 +
                                                  half * 2) = sc;
            } else if (2 * tl.nt + half < nblocks) {
#pragma unroll 2
                for (int j = 0; j < 8; ++j) {
                    uint32_t r[16];
                    tmem_ld16(lane_base + half * 128 + j * 16, r);
                    tmem_wait_ld(r);
                    if (valid) store16(args, row, tl.nt * kTN + half * 128 + j * 16, r);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&acc_empty));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <bool SW>
int launch(const Mx4Args &args, const void *a, cudaStream_t s) {
    auto kern = mx4_gemm_kernel<SW>;
    static std::once_flag once[64];
    static int rc[64];
    int dev = 0;
    MOE_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return cuda_fail("device ordinal beyond 63");
    std::call_once(once[dev], [&] {
        rc[dev] = (int)cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    });
    if (rc[dev]) return cuda_fail("cudaFuncSetAttribute", (cudaError_t)rc[dev]);
    CUtensorMap tmA, tmA32;
    if (!encode_2d_sw64(&tmA, a, (uint64_t)args.k_dim / 2, (uint64_t)args.rows, 128) ||
        !encode_2d_sw64(&tmA32, a, (uint64_t)args.k_dim / 2, (uint64_t)args.rows, 32))
        return cuda_fail("cuTensorMapEncodeTiled (activations)");
    const int64_t nt = ceil_div(args.n_out, kTN);
    const int64_t bound = nt * (args.groups + ceil_div(args.rows, kTM));
    const int grid = (int)std::min<int64_t>((int64_t)sm_count(), bound);
    return launch_dependent(kern, dim3(grid), dim3(kThreads), kSmemBytes, s, tmA, tmA32, args);
}

}  // namespace

int launch_mx4_gemm(int groups, int n_out, int k_dim, int rows, const void *a, const void *a_scales,
                    const int32_t *offsets, const void *w, const void *w_scales, void *c, int c_dtype,
                    int32_t *status, cudaStream_t s) {
    Mx4Args args = {};
    args.groups = groups;
    args.n_out = n_out;
    args.k_dim = k_dim;
    args.rows = rows;
    args.a_scales = static_cast<const uint8_t *>(a_scales);
    args.offsets = offsets;
    args.w = static_cast<const uint8_t *>(w);
    args.w_scales = static_cast<const uint8_t *>(w_scales);
    args.c = c;
    args.c_bf16 = c_dtype == MOE_OUT_BF16;
    args.status = status;
    return launch<false>(args, a, s);
}

int launch_mx4_gemm_swiglu(int groups, int inter, int k_dim, int rows, const void *a,
                           const void *a_scales, const int32_t *offsets, const void *w13,
                           const void *w13_scales, void *h, void *h_scales, int32_t *status,
                           cudaStream_t s) {
    Mx4Args args = {};
    args.groups = groups;
    args.n_out = 2 * inter;
    args.k_dim = k_dim;
    args.rows = rows;
    args.a_scales = static_cast<const uint8_t *>(a_scales);
    args.offsets = offsets;
    args.w = static_cast<const uint8_t *>(w13);
    args.w_scales = static_cast<const uint8_t *>(w13_scales);
    args.c = h;
    args.h_scales = static_cast<uint8_t *>(h_scales);
    args.status = status;
    return launch<true>(args, a, s);
}

}  // namespace moe
