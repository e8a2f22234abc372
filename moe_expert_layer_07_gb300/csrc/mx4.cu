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

// One thread takes eight elements, four neighbouring lanes a block.
template <bool F32>
__global__ void __launch_bounds__(kThreads)
    mx4_quantize_kernel(const void *__restrict__ in, uint32_t *__restrict__ codes,
                        uint8_t *__restrict__ scales, int64_t n8) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    // n8 is a multiple of 4, so the four lanes of a block leave together
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n8;
         i += (int64_t)gridDim.x * kThreads) {
        float v[8];
        if (F32) {
            const float4 a = __ldg(static_cast<const float4 *>(in) + 2 * i);
            const float4 b = __ldg(static_cast<const float4 *>(in) + 2 * i + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = __ldg(static_cast<const uint4 *>(in) + i);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
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

template <bool F32>
__global__ void __launch_bounds__(kThreads)
    mx4_dequantize_kernel(const uint32_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                          void *__restrict__ out, int64_t n8) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n8;
         i += (int64_t)gridDim.x * kThreads) {
        float v[8];
        mx4_values8(__ldg(codes + i), mx4_scale(__ldg(scales + (i >> 2))), v);
        if (F32) {
            float4 *o = static_cast<float4 *>(out) + 2 * i;
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {   // exact: an e2m1 value has two significant bits
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                w[j] = *reinterpret_cast<uint32_t *>(&b);
            }
            static_cast<uint4 *>(out)[i] = make_uint4(w[0], w[1], w[2], w[3]);
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

unsigned grid_for(int64_t n) {
    return (unsigned)std::min<int64_t>(ceil_div(n, kThreads), (int64_t)sm_count() * 16);
}

}  // namespace

int launch_mx4_quantize(int64_t rows, int64_t cols, const void *in, bool f32, void *codes,
                        void *scales, cudaStream_t s) {
    const int64_t n8 = rows * cols / 8;
    return launch_dependent(f32 ? mx4_quantize_kernel<true> : mx4_quantize_kernel<false>,
                            dim3(grid_for(n8)), dim3(kThreads), 0, s, in,
                            static_cast<uint32_t *>(codes), static_cast<uint8_t *>(scales), n8);
}

int launch_mx4_dequantize(int64_t rows, int64_t cols, const void *codes, const void *scales,
                          void *out, bool f32, cudaStream_t s) {
    const int64_t n8 = rows * cols / 8;
    return launch_dependent(f32 ? mx4_dequantize_kernel<true> : mx4_dequantize_kernel<false>,
                            dim3(grid_for(n8)), dim3(kThreads), 0, s,
                            static_cast<const uint32_t *>(codes),
                            static_cast<const uint8_t *>(scales), out, n8);
}

int launch_mx4_pack(int64_t groups, int64_t n_out, int64_t k_dim, const void *codes,
                    const void *scales, void *codes_t, void *scales_t, cudaStream_t s) {
    const int kt = (int)(k_dim / 128);
    const int64_t nrows = groups * n_out;
    return launch_dependent(mx4_pack_kernel, dim3(grid_for(nrows * kt * 4)), dim3(kThreads), 0, s,
                            static_cast<const uint4 *>(codes),
                            static_cast<const uint32_t *>(scales), static_cast<uint4 *>(codes_t),
                            static_cast<uint32_t *>(scales_t), nrows, kt);
}

}  // namespace moe
