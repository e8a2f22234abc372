// Products of 1 to 16 rows with weights in four bits:
//   y[t, n] = sum_k x[t, k] W[n, k]
// x in bf16, W in MXFP4 or as integers with group scales and zero points.
//
// Bound by reading W once: 4.25 bits a weight and more.  A warp takes 16 rows
// of W by a slice of 128 of K at a time, the M side of mma.sync m16n8k16, with
// 8 or 16 rows of x as its N side.  A slice of x stays in the warp's registers
// for all of its rows of W, so x costs nothing per weight: a CTA's warps share
// K among them, and where K is longer than a CTA's registers hold, the CTAs of a
// cluster do.  W comes by cp.async through a ring of each warp's own and leaves
// it by ldmatrix in the order of the products; scales go to registers, the next
// rows' ahead of their use.
//
// Codes become fp16 unscaled (MXFP4: cvt; integers: 1024 + code put together
// from bits, minus 1024 + zero point, both exact), products of 32 of K are
// multiplied by the group's scale in fp32.  x is fp16 times a power of two for
// each row (bf16 values have no more bits; below 2^-38 of a row's largest they
// lose some).
//
// Sums: the K slices of a warp one after the other, then warps in order, then
// CTAs in order: the same bits each time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "mx4.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kTileRows = 16, kSlice = 128;
constexpr int kTileBytes = kTileRows * kSlice / 2;
constexpr int kRingStages = 4;
constexpr int kHold = 16;   // row tiles whose sums a CTA of a cluster holds between exchanges

struct MatvecArgs {
    const uint16_t *x;
    const uint8_t *w;
    const void *scales;
    const uint8_t *zeros;
    void *y;
    int T, N, K, slices, warps, per_cta, group_shift, s_f32, out_bf16;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src))
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t sub_half2(uint32_t a, uint32_t b) {
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Scales of one slice of one row of W: four MXFP4 bytes, or as many group
// scales (raw bits) and zero points as the slice has.
struct RawScales {
    uint32_t s[4];   // MXFP4: s[0] the four bytes; integers: the scale of each block of 32
    uint32_t z;      // zero points of the four blocks
};

template <bool INT>
__device__ __forceinline__ RawScales load_scales(const MatvecArgs &a, int n, int slice) {
    RawScales r;
    r.z = 0x08080808u;
#pragma unroll
    for (int b = 0; b < 4; ++b) r.s[b] = 0;
    if (n >= a.N) return r;
    if (!INT) {
        const uint8_t *p = static_cast<const uint8_t *>(a.scales) + (int64_t)n * (a.K >> 5) + slice * 4;
        if ((a.K & 127) == 0) {
            r.s[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (slice * 4 + b < a.K >> 5) r.s[0] |= (uint32_t)__ldg(p + b) << (8 * b);
        }
    } else {
        const int groups = a.K >> a.group_shift, per = kSlice >> a.group_shift;   // 1, 2 or 4 a slice
        const int64_t at = (int64_t)n * groups;
        uint32_t z = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if (b >= per) break;
            const int gi = slice * per + b;
            uint32_t v = 0, zero = 8;
            if (gi < groups) {
                v = a.s_f32 ? __ldg(static_cast<const uint32_t *>(a.scales) + at + gi)
                            : (uint32_t)__ldg(static_cast<const uint16_t *>(a.scales) + at + gi) << 16;
                if (a.zeros) zero = __ldg(a.zeros + at + gi) & 15u;
            }
            // to the blocks of 32 that the group has
            if (per == 4) r.s[b] = v, z |= zero << (8 * b);
            else if (per == 2) {
                r.s[2 * b] = r.s[(2 * b + 1) & 3] = v;
                z |= zero * 0x0101u << (16 * b);
            } else {
                r.s[0] = r.s[1] = r.s[2] = r.s[3] = v;
                z = zero * 0x01010101u;
            }
        }
        r.z = z;
    }
    return r;
}

// Eight codes of one row (block b) as fp16 pairs (0,1) (2,3) (4,5) (6,7); integers in
// the order (0,4) (1,5) (2,6) (3,7), which x's fragments follow.
template <bool INT>
__device__ __forceinline__ void widen(uint32_t codes, uint32_t z, int b, uint32_t (&h)[4]) {
    if (!INT) {
        mx4_half8(codes, h);
    } else {
        const uint32_t one = 0x6400u + (z >> (8 * b) & 0xffu);   // 1024 + zero
        const uint32_t zz = one * 0x10001u;
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = sub_half2(((codes >> (4 * j)) & 0x000f000fu) | 0x64006400u, zz);
    }
}

// NQ: rows of x in eights.  S: slices of a warp.
template <bool INT, int NQ, int S>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) matvec4_kernel(const MatvecArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_up[16];   // what each row of x was multiplied by, undone
    __shared__ uint32_t s_max[16];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int rank = ptx::cluster_rank();
    const int ranks = a.slices > a.per_cta ? (a.slices + a.per_cta - 1) / a.per_cta : 1;
    const int cluster = blockIdx.x / ranks, clusters = gridDim.x / ranks;
    const int first_slice = rank * a.per_cta + warp * S;
    const int tiles = (a.N + kTileRows - 1) / kTileRows;
    const int mine = cluster < tiles ? (tiles - cluster + clusters - 1) / clusters : 0;
    uint8_t *ring = smem + warp * kRingStages * kTileBytes;
    const uint32_t ring_addr = ptx::smem_u32(ring);
    float *s_part = reinterpret_cast<float *>(smem + a.warps * kRingStages * kTileBytes);   // [2][warps][NQ * 128]
    float *s_hold = s_part + 2 * a.warps * NQ * 128;                                         // [kHold][NQ * 128]
    const int row_bytes = a.K >> 1;
    // Copies item i (tile i / S, slice i % S) into its slot of the ring
    auto fetch = [&](int i) {
        if (i < mine * S) {
            const int tile = cluster + i / S * clusters, slice = first_slice + i % S;
            const uint32_t slot = ring_addr + (i % kRingStages) * kTileBytes;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int p = 32 * j + lane, r = p >> 2, q = p & 3;
                const int n = tile * kTileRows + r;
                if (n < a.N && slice * 64 + q * 16 < row_bytes)
                    cp_async16(slot + r * 64 + ((q ^ ((r >> 1) & 3)) << 4),
                               a.w + (int64_t)n * row_bytes + slice * 64 + q * 16);
            }
        }
        cp_async_commit();
    };
    ptx::pdl_launch_dependents();
    // weights are constants of the program; x may be an earlier kernel's
    ptx::pdl_wait();
#pragma unroll
    for (int i = 0; i < kRingStages - 1; ++i) fetch(i);
    // pieces that lie behind K or N are never copied: their scales are zero, and
    // whatever bits the ring holds there are finite numbers
    if (tid < 16) s_max[tid] = 0;
    __syncthreads();
    // each row's largest magnitude, by each CTA over all of K
#pragma unroll 4
    for (int t = 0; t < a.T; ++t) {
        uint32_t m = 0;
        const uint4 *row = reinterpret_cast<const uint4 *>(a.x + (int64_t)t * a.K);
        for (int i = tid; i < a.K / 8; i += a.warps * 32) {
            const uint4 v = __ldg(row + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) m = max(m, max(w[j] << 16 & 0x7fff0000u, w[j] & 0x7fff0000u));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0 && m) atomicMax(s_max + t, m);
    }
    __syncthreads();
    // 2^up puts it into [2^14, 2^15); held where 2^up and 2^-up are numbers
    if (tid < 16) s_up[tid] = __uint_as_float((uint32_t)(min(max((int)(s_max[tid] >> 23), 27), 254) - 14) << 23);
    __syncthreads();
    uint32_t xf[S][8][NQ][2];   // slices, steps of 16, rows of x
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int t = 8 * n + g;
        const float f = __uint_as_float((254u << 23) - __float_as_uint(s_up[t]));   // 1 / s_up
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int k = (first_slice + i) * kSlice + 32 * b + 8 * c;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (t < a.T && k < a.K && first_slice + i < (rank + 1) * a.per_cta)
                    v = __ldg(reinterpret_cast<const uint4 *>(a.x + (int64_t)t * a.K + k));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                float e[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    e[2 * j] = __uint_as_float(w[j] << 16) * f;
                    e[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    xf[i][2 * b + j / 2][n][j & 1] = INT ? half2_bits(e[j], e[j + 4]) : half2_bits(e[2 * j], e[2 * j + 1]);
            }
    }
    const int mrow = (lane & 7) + ((lane >> 3) & 1) * 8, mblk = lane >> 4;
    RawScales nx[S][2];
    auto load_tile_scales = [&](int it) {
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const bool there = it < mine && first_slice + i < min(a.slices, (rank + 1) * a.per_cta);
                nx[i][r] = load_scales<INT>(a, there ? (cluster + it * clusters) * kTileRows + g + 8 * r : a.N,
                                            first_slice + i);
            }
    };
    load_tile_scales(0);

    for (int it = 0; it < mine; ++it) {
        RawScales cur[S][2];
#pragma unroll
        for (int i = 0; i < S; ++i) cur[i][0] = nx[i][0], cur[i][1] = nx[i][1];
        load_tile_scales(it + 1);
        float acc[NQ][4];
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int item = it * S + i;
            cp_async_wait<kRingStages - 2>();
            __syncwarp();
            fetch(item + kRingStages - 1);
            const uint32_t slot = ring_addr + (item % kRingStages) * kTileBytes;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t w[4];
                ldm4(slot + mrow * 64 + (((2 * x + mblk) ^ ((mrow >> 1) & 3)) << 4), w);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int b = 2 * x + y;
                    uint32_t w0[4], w1[4];
                    widen<INT>(w[2 * y], cur[i][0].z, b, w0);
                    widen<INT>(w[2 * y + 1], cur[i][1].z, b, w1);
                    const float f0 = INT ? __uint_as_float(cur[i][0].s[b]) : mx4_scale(cur[i][0].s[0] >> (8 * b) & 0xffu);
                    const float f1 = INT ? __uint_as_float(cur[i][1].s[b]) : mx4_scale(cur[i][1].s[0] >> (8 * b) & 0xffu);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma16816(d, w0[0], w1[0], w0[1], w1[1], xf[i][2 * b][n][0], xf[i][2 * b][n][1]);
                        mma16816(d, w0[2], w1[2], w0[3], w1[3], xf[i][2 * b + 1][n][0], xf[i][2 * b + 1][n][1]);
                        acc[n][0] = fmaf(d[0], f0, acc[n][0]);
                        acc[n][1] = fmaf(d[1], f0, acc[n][1]);
                        acc[n][2] = fmaf(d[2], f1, acc[n][2]);
                        acc[n][3] = fmaf(d[3], f1, acc[n][3]);
                    }
                }
            }
        }
        // the warps' sums of this tile: [row of W][row of x]
        float *part = s_part + (it & 1) * a.warps * NQ * 128;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float *p = part + warp * NQ * 128 + 8 * n + 2 * c;
            *reinterpret_cast<float2 *>(p + g * 8 * NQ) = make_float2(acc[n][0], acc[n][1]);
            *reinterpret_cast<float2 *>(p + (g + 8) * 8 * NQ) = make_float2(acc[n][2], acc[n][3]);
        }
        // one barrier a tile: `part` is written again two tiles on, past the next one
        __syncthreads();
        for (int i = tid; i < NQ * 128; i += a.warps * 32) {
            float v = 0.0f;
            for (int w = 0; w < a.warps; ++w) v += part[w * NQ * 128 + i];
            const int t = i & (8 * NQ - 1), n = (cluster + it * clusters) * kTileRows + i / (8 * NQ);
            if (ranks > 1) {
                s_hold[(it % kHold) * NQ * 128 + i] = v;
            } else if (t < a.T && n < a.N) {
                v *= s_up[t];
                if (a.out_bf16) static_cast<__nv_bfloat16 *>(a.y)[(int64_t)t * a.N + n] = __float2bfloat16(v);
                else static_cast<float *>(a.y)[(int64_t)t * a.N + n] = v;
            }
        }
        if (ranks > 1 && (it % kHold == kHold - 1 || it == mine - 1)) {
            // the CTAs' sums together: CTA r finishes its share of what is held
            const int held = it % kHold + 1, base = it - it % kHold;
            ptx::cluster_sync();
            const uint32_t mem = ptx::smem_u32(s_hold);
            for (int i = rank * a.warps * 32 + tid; i < held * NQ * 128; i += ranks * a.warps * 32) {
                float v = 0.0f;
                for (int r = 0; r < ranks; ++r) {
                    float p;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p) : "r"(ptx::cluster_map(mem + 4 * i, r)));
                    v += p;
                }
                const int j = i % (NQ * 128), t = j & (8 * NQ - 1);
                const int n = (cluster + (base + i / (NQ * 128)) * clusters) * kTileRows + j / (8 * NQ);
                if (t < a.T && n < a.N) {
                    v *= s_up[t];
                    if (a.out_bf16) static_cast<__nv_bfloat16 *>(a.y)[(int64_t)t * a.N + n] = __float2bfloat16(v);
                    else static_cast<float *>(a.y)[(int64_t)t * a.N + n] = v;
                }
            }
            ptx::cluster_sync();   // nobody reads this CTA's shared memory any more
        }
    }
    cp_async_wait<0>();
}

template <bool INT, int NQ, int S>
int launch(const MatvecArgs &a, int ranks, int clusters, cudaStream_t s) {
    const int smem = a.warps * kRingStages * kTileBytes + (2 * a.warps + kHold) * NQ * 128 * 4;
    MOE_CUDA_TRY(cudaFuncSetAttribute(matvec4_kernel<INT, NQ, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(ranks * clusters));
    c.blockDim = dim3((unsigned)(a.warps * 32));
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)ranks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&c, matvec4_kernel<INT, NQ, S>, (const MatvecArgs)a);
    return e == cudaSuccess ? MOE_OK : cuda_fail("cudaLaunchKernelEx", e);
}

}  // namespace

int launch_w4_matvec(const moe_w4 *d, int T, const void *x, const void *codes, const void *scales,
                     const void *zeros, void *y, int out_dtype, cudaStream_t s) {
    MatvecArgs a;
    a.x = static_cast<const uint16_t *>(x);
    a.w = static_cast<const uint8_t *>(codes);
    a.scales = scales;
    a.zeros = static_cast<const uint8_t *>(zeros);
    a.y = y;
    a.T = T;
    a.N = d->n_out;
    a.K = d->k_dim;
    a.slices = (int)ceil_div(a.K, kSlice);
    a.group_shift = d->group == 32 ? 5 : d->group == 64 ? 6 : 7;
    a.s_f32 = d->scale_dtype == MOE_OUT_F32;
    a.out_bf16 = out_dtype == MOE_OUT_BF16;
    // Slices a warp and CTAs a cluster: x's registers are 16 (8 rows) or 32 a slice
    const int per_warp = a.slices > kMaxWarps ? 2 : 1;
    int ranks = 1;
    while (ranks * kMaxWarps * per_warp < a.slices) ranks *= 2;   // 32768 of K: 8
    a.warps = (int)ceil_div(ceil_div(a.slices, ranks), per_warp);
    a.per_cta = a.warps * per_warp;
    ranks = (int)ceil_div(a.slices, a.per_cta);
    const int tiles = (int)ceil_div(a.N, kTileRows);
    const int clusters = std::max(1, std::min(tiles, sm_count() / ranks));
    const bool i = d->kind == MOE_W4_INT, wide = T > 8;
    if (per_warp == 1) {
        if (i) return wide ? launch<true, 2, 1>(a, ranks, clusters, s) : launch<true, 1, 1>(a, ranks, clusters, s);
        return wide ? launch<false, 2, 1>(a, ranks, clusters, s) : launch<false, 1, 1>(a, ranks, clusters, s);
    }
    if (i) return wide ? launch<true, 2, 2>(a, ranks, clusters, s) : launch<true, 1, 2>(a, ranks, clusters, s);
    return wide ? launch<false, 2, 2>(a, ranks, clusters, s) : launch<false, 1, 2>(a, ranks, clusters, s);
}

}  // namespace moe
