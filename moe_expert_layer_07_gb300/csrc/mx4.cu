// MXFP4 (OCP microscaling, e2m1 elements): quantisation, its inverse, and
// the tile packing of expert weights.
//
// A block is 32 consecutive elements of a row.  With m its largest magnitude
//   e    = max(floor(log2 m) - 2, -127)       (2 = the exponent of e2m1's 6)
//   code = e2m1(v / 2^e), round to nearest even, saturating at 6
// and the scale byte is e + 127 (ue8m0).  A block of zeros has e = 0; a block
// with an infinity or a NaN has the byte 255, which stands for NaN, and zero
// codes.  Division by a power of two is exact, so the codes do not depend on
// the order of anything.  Two codes to a byte, the even element in the low
// half.
//
// Bound by memory: 2 or 4 bytes an element on one side, 4.25 bits on the other.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "mx4.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// One thread takes eight elements, four neighbouring lanes a block; U of them
// at a time, one CTA's width apart, so that enough loads are under way.
template <bool F32, int U>
__global__ void __launch_bounds__(kThreads)
    mx4_quantize_kernel(const void *__restrict__ in, uint32_t *__restrict__ codes,
                        uint8_t *__restrict__ scales, int64_t n8) {
    constexpr int W = F32 ? 2 : 1;   // 16-byte pieces of eight elements
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    // n8 is a multiple of 4, so the four lanes of a block leave together
    for (int64_t i0 = (int64_t)blockIdx.x * (kThreads * U) + threadIdx.x; i0 < n8;
         i0 += (int64_t)gridDim.x * (kThreads * U)) {
        uint4 raw[U][W];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int w = 0; w < W; ++w)
                if (i0 + u * kThreads < n8)
                    raw[u][w] = __ldg(static_cast<const uint4 *>(in) + (i0 + u * kThreads) * W + w);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * kThreads;
            if (i >= n8) break;
            float v[8];
            const uint32_t w[4] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w};
            if (F32) {
                const uint4 q = raw[u][W - 1];
                const uint32_t x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(w[j]), v[4 + j] = __uint_as_float(x[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] = __uint_as_float(w[j] << 16);
                    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                }
            }
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
            const uint32_t quad = 0xfu << (threadIdx.x & 28);
            m = max(m, __shfl_xor_sync(quad, m, 1));
            m = max(m, __shfl_xor_sync(quad, m, 2));
            const uint32_t byte = mx4_scale_byte(m);
            codes[i] = mx4_codes8(v, byte);
            if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
        }
    }
}

// A thread writes 16 bytes at a time, its neighbours the next: four fp32 or
// eight bf16 values.
template <bool F32, int U>
__global__ void __launch_bounds__(kThreads)
    mx4_dequantize_kernel(const void *__restrict__ codes, const uint8_t *__restrict__ scales,
                          uint4 *__restrict__ out, int64_t n) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    for (int64_t i0 = (int64_t)blockIdx.x * (kThreads * U) + threadIdx.x; i0 < n;
         i0 += (int64_t)gridDim.x * (kThreads * U)) {
        uint32_t c[U], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * kThreads;
            if (i >= n) continue;
            c[u] = F32 ? __ldg(static_cast<const uint16_t *>(codes) + i)
                       : __ldg(static_cast<const uint32_t *>(codes) + i);
            s[u] = __ldg(scales + (i >> (F32 ? 3 : 2)));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * kThreads;
            if (i >= n) break;
            float v[8];
            mx4_values8(c[u], mx4_scale(s[u]), v);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (F32) {
                    w[j] = __float_as_uint(v[j]);
                } else {   // exact: an e2m1 value has two significant bits
                    __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    w[j] = *reinterpret_cast<uint32_t *>(&b);
                }
            }
            ptx::store_past_l1(out + i, make_uint4(w[0], w[1], w[2], w[3]));   // 2048 rows: 7.3 -> 6.4 us
        }
    }
}

// Codes [groups, n_out, k/2] -> 128 x 64-byte tiles, tile-major; chunk c (16
// bytes) of row r at position c ^ ((r / 2) mod 4).  Scales [groups, n_out,
// k/32] -> 512 bytes a tile, byte (r mod 32) 16 + (r / 32) 4 + j for block j.
__global__ void __launch_bounds__(kThreads)
    mx4_pack_kernel(const uint4 *__restrict__ codes, const uint32_t *__restrict__ scales,
                    uint4 *__restrict__ codes_t, uint32_t *__restrict__ scales_t, int64_t nrows,
                    int kt) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int64_t n = nrows * kt * 4;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * kThreads) {
        // written in order: position p of row r of tile `tile`
        const int64_t tile = i >> 9;
        const int r = (int)(i >> 2) & 127, p = (int)i & 3, c = p ^ ((r >> 1) & 3);
        const int64_t row = tile / kt * 128 + r;
        const int kb = (int)(tile % kt);
        codes_t[i] = __ldg(codes + (row * kt + kb) * 4 + c);
        if (p == 0)
            scales_t[tile * 128 + (r & 31) * 4 + (r >> 5)] = __ldg(scales + row * kt + kb);
    }
}

// Large calls have four chunks a thread under way: 16384 rows of 7168 bf16
// quantise in 48.6 us (6.1 TB/s; 50.4 with one) and read back in 44.6 (6.7;
// 48.8 with one), fp32 in 77.2 (6.9 TB/s) and 81.3 (6.5).  Small ones spread over as many threads as they have chunks.
constexpr int kDeep = 4;
bool deep(int64_t n) { return n >= (int64_t)kDeep * kThreads * sm_count() * 8; }

// Quantising, a loop over 16 CTAs an SM measured faster than one CTA a piece
// (48.6 against 49.3 us), reading back the other way (48.6 against 44.6).
unsigned grid_for(int64_t n, bool looped) {
    const int64_t all = ceil_div(n, kThreads), most = looped ? (int64_t)sm_count() * 16 : INT32_MAX;
    return (unsigned)std::min(all, most);
}

}  // namespace

int launch_mx4_quantize(int64_t rows, int64_t cols, const void *in, bool f32, void *codes,
                        void *scales, cudaStream_t s) {
    const int64_t n8 = rows * cols / 8;
    const bool d = deep(n8);
    auto kern = f32 ? (d ? mx4_quantize_kernel<true, kDeep> : mx4_quantize_kernel<true, 1>)
                    : (d ? mx4_quantize_kernel<false, kDeep> : mx4_quantize_kernel<false, 1>);
    return launch_dependent(kern, dim3(grid_for(d ? ceil_div(n8, kDeep) : n8, true)), dim3(kThreads), 0, s,
                            in, static_cast<uint32_t *>(codes), static_cast<uint8_t *>(scales), n8);
}

int launch_mx4_dequantize(int64_t rows, int64_t cols, const void *codes, const void *scales,
                          void *out, bool f32, cudaStream_t s) {
    const int64_t n = rows * cols / (f32 ? 4 : 8);
    const bool d = deep(n);
    auto kern = f32 ? (d ? mx4_dequantize_kernel<true, kDeep> : mx4_dequantize_kernel<true, 1>)
                    : (d ? mx4_dequantize_kernel<false, kDeep> : mx4_dequantize_kernel<false, 1>);
    return launch_dependent(kern, dim3(grid_for(d ? ceil_div(n, kDeep) : n, false)), dim3(kThreads), 0, s,
                            codes, static_cast<const uint8_t *>(scales), static_cast<uint4 *>(out), n);
}

int launch_mx4_pack(int64_t groups, int64_t n_out, int64_t k_dim, const void *codes,
                    const void *scales, void *codes_t, void *scales_t, cudaStream_t s) {
    const int kt = (int)(k_dim / 128);
    const int64_t nrows = groups * n_out;
    return launch_dependent(mx4_pack_kernel, dim3(grid_for(nrows * kt * 4, true)), dim3(kThreads), 0, s,
                            static_cast<const uint4 *>(codes),
                            static_cast<const uint32_t *>(scales), static_cast<uint4 *>(codes_t),
                            static_cast<uint32_t *>(scales_t), nrows, kt);
}

}  // namespace moe
