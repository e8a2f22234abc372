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
// (r', x).  One CTA holds one row in registers, at most VPT chunks of eight
// elements a thread, so both norms work on registers; y and r stay in their
// own type until they are used, which keeps enough CTAs on an SM to have the
// next rows' loads in flight while these reduce.  Layer norm subtracts the
// mean before it squares, also in registers, instead of taking E[v^2] -
// mean^2, which cancels.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

struct NormArgs {
    const void *y, *r, *gate, *w_post, *b_post, *w_pre, *b_pre;
    void *r_out;
    uint16_t *x_out;
    int T, H;
    int p_f32, gate_mode, layer;
    float eps, rs, bs;
};

// Pairs of fp32 numbers in one register pair: the packed instructions do two
// elements each (the unpaired ones made this kernel issue-bound at bf16).
using F2 = uint64_t;
__device__ __forceinline__ F2 pair(float lo, float hi) {
    return ptx::pack2(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float lo2(F2 v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(F2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Eight elements as they lie in memory, and as pairs.
template <bool F32>
struct Raw {
    uint4 a[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p, size_t i) {
#pragma unroll
        for (int j = 0; j < (F32 ? 2 : 1); ++j)
            a[j] = static_cast<const uint4 *>(p)[(F32 ? 2 : 1) * i + j];
    }
    // What a row is read once for, past L1 (16384 bf16 rows of 7168: 151 -> 146
    // us with its stores; layer norm 207 -> 190).  Not fp32, whose two pieces
    // share a sector (261 -> 270).
    __device__ __forceinline__ void load_once(const void *p, size_t i) {
        if (F32) load(p, i);
        else a[0] = ptx::load_past_l1(static_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void get(F2 (&v)[4]) const {
        if (F32) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint4 q = a[F32 ? j : 0];
                v[2 * j] = ptx::pack2(q.x, q.y);
                v[2 * j + 1] = ptx::pack2(q.z, q.w);
            }
        } else {
            const uint32_t w[4] = {a[0].x, a[0].y, a[0].z, a[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = ptx::pack2(w[j] << 16, w[j] & 0xffff0000u);
        }
    }
};

__device__ __forceinline__ void load8(const void *p, int f32, size_t i, F2 (&v)[4]) {
    if (f32) {
        Raw<true> r;
        r.load(p, i);
        r.get(v);
    } else {
        Raw<false> r;
        r.load(p, i);
        r.get(v);
    }
}

template <bool F32>
__device__ __forceinline__ void store8(void *p, size_t i, const F2 (&v)[4]) {
    if (F32) {
        float4 *o = static_cast<float4 *>(p) + 2 * i;
        o[0] = make_float4(lo2(v[0]), hi2(v[0]), lo2(v[1]), hi2(v[1]));
        o[1] = make_float4(lo2(v[2]), hi2(v[2]), lo2(v[3]), hi2(v[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            __nv_bfloat162 b = __floats2bfloat162_rn(lo2(v[j]), hi2(v[j]));
            w[j] = *reinterpret_cast<uint32_t *>(&b);
        }
        ptx::store_past_l1(static_cast<uint4 *>(p) + i, make_uint4(w[0], w[1], w[2], w[3]));
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

// The (negated) mean and the inverse size of a row: norm(v) = (v - mean) inv.
// get(i, v) gives chunk i of this thread (false past the row's end).
template <int VPT, bool LAYER, typename Get>
__device__ __forceinline__ float2 row_stats(const NormArgs &a, Get get, float (*sh)[32], int &slot) {
    const float inv_h = 1.0f / (float)a.H;
    F2 v[4], s = 0ull;
    float mean = 0.0f;
    if (LAYER) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (get(i, v))
#pragma unroll
                for (int j = 0; j < 4; ++j) s = add2(s, v[j]);
        mean = block_sum(lo2(s) + hi2(s), sh, slot) * inv_h;
        s = 0ull;
    }
    const F2 m = pair(-mean, -mean);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (get(i, v))
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const F2 d = LAYER ? add2(v[j], m) : v[j];
                s = ptx::fma2(d, d, s);
            }
    return make_float2(-mean, rsqrtf(block_sum(lo2(s) + hi2(s), sh, slot) * inv_h + a.eps));
}

// (v - mean) inv w (+ b) for chunk c of the row
template <bool LAYER>
__device__ __forceinline__ void apply(F2 (&v)[4], const NormArgs &a, float2 st, const void *w,
                                      const void *b, int c) {
    F2 p[4];
    load8(w, a.p_f32, c, p);
    const F2 m = pair(st.x, st.x), inv = pair(st.y, st.y);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul2(mul2(LAYER ? add2(v[j], m) : v[j], inv), p[j]);
    if (b) {
        load8(b, a.p_f32, c, p);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = add2(v[j], p[j]);
    }
}

// blockDim = (threads of a row, rows): a CTA takes several rows only if a warp
// holds a whole row.
template <int VPT, bool Y32, bool R32, bool LAYER>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : VPT == 2 ? 512 : 256, VPT == 4 ? 4 : 1) block_norm_kernel(const NormArgs a) {
    __shared__ float sh[2][32];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();   // the block's output of an earlier kernel
    const int n8 = a.H >> 3;
    const size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= (size_t)a.T) return;   // whole warps, or the CTA
    const size_t base = row * n8;
    int slot = 0;
    Raw<Y32> y[VPT];
    Raw<R32> r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < n8) {
            if (a.y) y[i].load_once(a.y, base + c);
            r[i].load_once(a.r, base + c);
            // wanted after the first reduction (16384 bf16 rows of 7168: 220 -> 184 us)
            if (a.gate_mode == MOE_GATE_FULL)
                ptx::prefetch_l2_line(static_cast<const uint4 *>(a.gate) + (base + c) * (a.p_f32 ? 2 : 1));
        }
    }
    float2 st = make_float2(0.0f, 1.0f);
    if (a.w_post)
        st = row_stats<VPT, LAYER>(a, [&](int i, F2 (&v)[4]) {
            if ((int)(threadIdx.x + i * blockDim.x) >= n8) return false;
            y[i].get(v);
            return true;
        }, sh, slot);
    F2 rs = pair(a.rs, a.rs), bs = pair(a.bs, a.bs);
    if (a.gate_mode == MOE_GATE_TOKEN) {
        const float g = a.p_f32 ? static_cast<const float *>(a.gate)[row]
                                : __uint_as_float((uint32_t)static_cast<const uint16_t *>(a.gate)[row] << 16);
        bs = pair(a.bs * g, a.bs * g);
    }
    F2 x[VPT][4];   // r', unrounded
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= n8) continue;
        r[i].get(x[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = mul2(rs, x[i][j]);
        if (a.y) {
            F2 n[4];
            y[i].get(n);
            if (a.w_post) apply<LAYER>(n, a, st, a.w_post, a.b_post, c);
            if (a.gate_mode == MOE_GATE_FEATURE || a.gate_mode == MOE_GATE_FULL) {
                F2 g[4];
                load8(a.gate, a.p_f32, a.gate_mode == MOE_GATE_FEATURE ? (size_t)c : base + c, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) n[j] = mul2(n[j], g[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] = ptx::fma2(bs, n[j], x[i][j]);
        }
        if (a.r_out) store8<R32>(a.r_out, base + c, x[i]);
    }
    if (!a.x_out) return;
    st = row_stats<VPT, LAYER>(a, [&](int i, F2 (&v)[4]) {
        if ((int)(threadIdx.x + i * blockDim.x) >= n8) return false;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = x[i][j];
        return true;
    }, sh, slot);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= n8) continue;
        apply<LAYER>(x[i], a, st, a.w_pre, a.b_pre, c);
        store8<false>(a.x_out, base + c, x[i]);
    }
}

template <int VPT, bool Y32, bool R32>
int launch_rows(const NormArgs &a, cudaStream_t s) {
    auto kern = a.layer ? block_norm_kernel<VPT, Y32, R32, true> : block_norm_kernel<VPT, Y32, R32, false>;
    const unsigned threads = (unsigned)(ceil_div(ceil_div(a.H / 8, VPT), 32) * 32);
    const unsigned rows = threads == 32 ? 8 : 1;
    return launch_dependent(kern, dim3((unsigned)ceil_div(a.T, rows)), dim3(threads, rows), 0, s, a);
}

template <bool Y32, bool R32>
int launch_typed(const NormArgs &a, cudaStream_t s) {
    const int n8 = a.H / 8;
    // Threads a row.  Few rows: one chunk a thread, the shortest chain (7 rows
    // of 7168: 3.2 us, four chunks a thread 5.0).  Many rows: enough rows on an
    // SM at once to cover one another's reductions, and few threads to reduce
    // over (16384 rows of 7168 bf16: 317 / 190 / 152 us with 1 / 2 / 4 chunks;
    // fp32 rows, whose chunks take twice the registers: 371 / 263 / 326; of
    // 1024 bf16: 30 / 26 / 28; 65536 rows of 256: 28 / 32 / 36; all while bf16
    // rows went through L1, past it the first is 147 with 4).
    // Above 8192 columns one shape, eight chunks on 256 threads, takes all calls.
    // It is the better one for many bf16 rows alone: 16384 columns, against two
    // chunks on 1024 threads, 4096 bf16 rows 101 / 125 us, fp32 276 / 173, 7 rows
    // 8.6 / 4.7; 12288 columns 93 / 104, 232 / 142, 8.4 / 4.2.
    if (n8 > 1024) return launch_rows<8, Y32, R32>(a, s);
    if (a.T <= 2 * sm_count() || n8 <= 64) return launch_rows<1, Y32, R32>(a, s);
    if (n8 <= 512 || Y32 || R32) return launch_rows<2, Y32, R32>(a, s);
    return launch_rows<4, Y32, R32>(a, s);
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
    a.T = T;
    a.H = d->hidden;
    a.p_f32 = d->param_dtype == MOE_OUT_F32;
    a.gate_mode = d->gate_mode;
    a.layer = d->kind == MOE_NORM_LAYER;
    a.eps = d->eps;
    a.rs = d->residual_scale;
    a.bs = d->branch_scale;
    const bool y32 = d->y_dtype == MOE_OUT_F32, r32 = d->residual_dtype == MOE_OUT_F32;
    if (y32) return r32 ? launch_typed<true, true>(a, s) : launch_typed<true, false>(a, s);
    return r32 ? launch_typed<false, true>(a, s) : launch_typed<false, false>(a, s);
}

}  // namespace moe
