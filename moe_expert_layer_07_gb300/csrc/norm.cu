// The norms before and after a block, with the block's gate and residual
// scale, in one pass over the rows:
//
//   n  = post ? norm(y) w_post (+ b_post) : y
//   r' = residual_scale r + branch_scale gate n
//   x  = norm(r') w_pre (+ b_pre)
//
// norm(v) = v / sqrt(mean(v^2) + eps) (RMS), or with the mean taken off first
// (layer norm).  y is a block's output (NULL: r' = residual_scale r), r the
// residual stream, r' its new value, x the next block's input.  Everything is
// fp32 from load to store; r' and x are rounded once, and x is formed from
// the unrounded r'.
//
// Bound by memory: a row is read once (y, r, the full gate) and written once
// (r', x).  One CTA holds one row in registers (at most VPT chunks of eight
// elements a thread), so both norms work on registers; layer norm subtracts
// the mean before it squares, also in registers, instead of taking
// E[v^2] - mean^2, which cancels.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

struct NormArgs {
    const void *y, *r, *gate, *w_post, *b_post, *w_pre, *b_pre;
    void *r_out;
    uint16_t *x_out;
    int H;
    int y_f32, r_f32, p_f32, gate_mode, layer;
    float eps, rs, bs;
};

__device__ __forceinline__ void load8(const void *p, int f32, size_t i, float (&v)[8]) {
    if (f32) {
        const float4 a = reinterpret_cast<const float4 *>(p)[2 * i];
        const float4 b = reinterpret_cast<const float4 *>(p)[2 * i + 1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = reinterpret_cast<const uint4 *>(p)[i];
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ void store8(void *p, int f32, size_t i, const float (&v)[8]) {
    if (f32) {
        reinterpret_cast<float4 *>(p)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<uint32_t *>(&b);
        }
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Sum over the CTA; `slot` alternates between calls so that one barrier a
// call is enough (a slot is rewritten two calls later, past that barrier).
__device__ __forceinline__ float block_sum(float v, float (*sh)[32], int &slot) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    float *s = sh[slot];
    slot ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = (threadIdx.x & 31) < nw ? s[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
}

// v -> norm(v) w (+ b) for this thread's chunks of the row
template <int VPT>
__device__ __forceinline__ void normalise(float (&v)[VPT][8], const NormArgs &a, const void *w,
                                          const void *b, int n8, float (*sh)[32], int &slot) {
    const float inv_h = 1.0f / (float)a.H;
    float mean = 0.0f;
    if (a.layer) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j];
        mean = block_sum(s, sh, slot) * inv_h;
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if ((int)(threadIdx.x + i * blockDim.x) >= n8) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[i][j] -= mean;
            ss = fmaf(v[i][j], v[i][j], ss);
        }
    }
    const float inv = rsqrtf(block_sum(ss, sh, slot) * inv_h + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= n8) continue;
        float wv[8];
        load8(w, a.p_f32, c, wv);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * inv * wv[j];
        if (b) {
            load8(b, a.p_f32, c, wv);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += wv[j];
        }
    }
}

template <int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 256) block_norm_kernel(const NormArgs a) {
    __shared__ float sh[2][32];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();   // the block's output of an earlier kernel
    const int n8 = a.H >> 3;
    const size_t row = blockIdx.x, base = row * (size_t)n8;
    int slot = 0;
    // chunks past the row's end stay zero: they add nothing to a sum
    float n[VPT][8], r[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
        for (int j = 0; j < 8; ++j) n[i][j] = r[i][j] = 0.0f;
        if (c < n8) {
            if (a.y) load8(a.y, a.y_f32, base + c, n[i]);
            load8(a.r, a.r_f32, base + c, r[i]);
        }
    }
    if (a.w_post) normalise<VPT>(n, a, a.w_post, a.b_post, n8, sh, slot);
    float tok_gate = 1.0f;
    if (a.gate_mode == MOE_GATE_TOKEN)
        tok_gate = a.p_f32 ? static_cast<const float *>(a.gate)[row]
                           : __uint_as_float((uint32_t)static_cast<const uint16_t *>(a.gate)[row] << 16);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= n8) continue;
        if (a.y) {
            float g[8];
            if (a.gate_mode == MOE_GATE_FEATURE) load8(a.gate, a.p_f32, c, g);
            else if (a.gate_mode == MOE_GATE_FULL) load8(a.gate, a.p_f32, base + c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v = n[i][j];
                if (a.gate_mode == MOE_GATE_TOKEN) v *= tok_gate;
                else if (a.gate_mode != MOE_GATE_NONE) v *= g[j];
                r[i][j] = fmaf(a.bs, v, a.rs * r[i][j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] *= a.rs;
        }
        if (a.r_out) store8(a.r_out, a.r_f32, base + c, r[i]);
    }
    if (!a.x_out) return;
    normalise<VPT>(r, a, a.w_pre, a.b_pre, n8, sh, slot);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < n8) store8(a.x_out, 0, base + c, r[i]);
    }
}

}  // namespace

int launch_block_norm(const moe_norm *d, int T, const void *y, const void *residual,
                      const void *gate, const void *w_post, const void *b_post,
                      const void *w_pre, const void *b_pre, void *residual_out, void *x_out,
                      cudaStream_t s) {
    NormArgs a;
    a.y = y;
    a.r = residual;
    a.gate = gate;
    a.w_post = w_post;
    a.b_post = b_post;
    a.w_pre = w_pre;
    a.b_pre = b_pre;
    a.r_out = residual_out;
    a.x_out = static_cast<uint16_t *>(x_out);
    a.H = d->hidden;
    a.y_f32 = d->y_dtype == MOE_OUT_F32;
    a.r_f32 = d->residual_dtype == MOE_OUT_F32;
    a.p_f32 = d->param_dtype == MOE_OUT_F32;
    a.gate_mode = d->gate_mode;
    a.layer = d->kind == MOE_NORM_LAYER;
    a.eps = d->eps;
    a.rs = d->residual_scale;
    a.bs = d->branch_scale;
    const int n8 = d->hidden / 8;
    auto threads = [&](int vpt) { return (unsigned)(ceil_div(ceil_div(n8, vpt), 32) * 32); };
    if (n8 <= 1024)
        return launch_dependent(block_norm_kernel<4>, dim3(T), dim3(threads(4)), 0, s, a);
    return launch_dependent(block_norm_kernel<8>, dim3(T), dim3(threads(8)), 0, s, a);
}

}  // namespace moe
