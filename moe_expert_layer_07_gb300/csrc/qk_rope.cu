// Norm of queries and keys for each head, the rotation by the token's position,
// and the write of keys and values into the four-bit cache, in one pass.
//
//   n = v / sqrt(mean(v^2) + eps) w
//   a, b -> a cos - b sin, b cos + a sin      (the pairs of the first R channels)
//
// A head is dim / 8 neighbouring lanes of eight channels: the norm's sum and the
// block maxima of MXFP4 are butterflies over them.  Where pairs are half a
// rotation apart a lane takes four channels and their four partners.
// Everything is fp32 until the one rounding of each output; keys go to four
// bits not by way of bf16, from sums of two fp32 numbers.
//
// Bound by memory, and by the issue of instructions nearly as much: a row is read and
// written once.  A warp keeps one token's angles in registers over the heads that it
// takes, the next ones' loads under way.  Keys for the cache, five times a query's
// work, have rounds of their own, the first ones (last, they were what a warp ended
// with: 5001 rows 17.9 us for 16.4).  Measured: 8192 rows of 64 + 16 heads of 128 51.4 us
// (5.95 TB/s), into the cache 74 (4.2); 5001 rows of 32 + 8 heads of 64 into the
// cache 16.4 us (2.9 TB/s: two waves of warps, 4 us of it launch and end); 7 rows 2.3
// in a graph, 6.5 where the call is the host's.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "mx4.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
    const uint16_t *qkv;
    const int32_t *positions;
    const float *cos_sin;
    const void *w_q, *w_k;
    uint16_t *q_out, *k_out;
    uint16_t *codes;
    uint8_t *scales;
    const int32_t *slots;
    int32_t *status;
    int64_t stride, slots_in_cache;
    int T, parts, Hq, Hk, R, w_f32, max_positions, page_shift;   // parts: warps that share a row
    float eps;
};

// Pairs of fp32 numbers: the packed instructions do two channels each.
using F2 = uint64_t;
__device__ __forceinline__ F2 pair(float lo, float hi) { return ptx::pack2(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float lo2(F2 v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(F2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
using ptx::mul2;

__device__ __forceinline__ uint2 load_once(const uint16_t *p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
// Four channels as two pairs
__device__ __forceinline__ void unpack4(const uint2 q, F2 (&v)[2]) {
    v[0] = ptx::pack2(q.x << 16, q.x & 0xffff0000u);
    v[1] = ptx::pack2(q.y << 16, q.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(uint16_t *p, const F2 (&v)[2]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(lo2(v[0]), hi2(v[0])), b = __floats2bfloat162_rn(lo2(v[1]), hi2(v[1]));
    asm volatile("st.global.L1::no_allocate.v2.b32 [%0], {%1, %2};" ::"l"(p),
                 "r"(*reinterpret_cast<const uint32_t *>(&a)), "r"(*reinterpret_cast<const uint32_t *>(&b))
                 : "memory");
}
__device__ __forceinline__ void load_w(const float *w, F2 (&v)[2]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(w);
    v[0] = ptx::pack2(a.x, a.y), v[1] = ptx::pack2(a.z, a.w);
}

// Pairs, exactly: a + b = hi + lo, a b = hi + lo
__device__ __forceinline__ F2 sub2(F2 a, F2 b) { return ptx::fma2(b, 0xbf800000bf800000ull, a); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return ptx::fma2(b, 0x3f8000003f800000ull, a); }
__device__ __forceinline__ F2 swapped(F2 v) { return pair(hi2(v), lo2(v)); }
__device__ __forceinline__ void two_sum(F2 a, F2 b, F2 &hi, F2 &lo) {
    hi = add2(a, b);
    const F2 z = sub2(hi, a);
    lo = add2(sub2(a, sub2(hi, z)), sub2(b, z));
}
__device__ __forceinline__ void two_product(F2 a, F2 b, F2 &hi, F2 &lo) {
    hi = mul2(a, b);
    lo = ptx::fma2(a, b, hi ^ 0x8000000080000000ull);
}
__device__ __forceinline__ void two_sum(float a, float b, float &hi, float &lo) {
    hi = a + b;
    const float z = hi - a;
    lo = (a - (hi - z)) + (b - z);
}

// A lane's channels of a key (v), normed and turned, v + lo: some 2^-44 off, so that codes are those of
// exact values.  (fp32's own error put one code in ten million on the other side of a border.)
// w: the norm's weights or NULL; cs, sn: as the kernel has them.
template <int D, bool PAIRS>
__device__ __forceinline__ void key_values(F2 (&v)[4], F2 (&lo)[4], const float *w, int ch_a, int ch_b, float eps, bool turned,
                                           const F2 (&cs)[PAIRS ? 4 : 2], const F2 (&sn)[PAIRS ? 4 : 2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) lo[i] = 0ull;
    if (w) {
        F2 s2 = mul2(v[0], v[0]), l2 = 0ull, e2;   // squares of bf16 numbers are exact
#pragma unroll
        for (int i = 1; i < 4; ++i) two_sum(s2, mul2(v[i], v[i]), s2, e2), l2 = add2(l2, e2);
        float s, sl, e;
        two_sum(lo2(s2), hi2(s2), s, e);
        sl = (lo2(l2) + hi2(l2)) + e;
#pragma unroll
        for (int o = D / 16; o >= 1; o >>= 1) {
            const float os = __shfl_xor_sync(0xffffffffu, s, o), ol = __shfl_xor_sync(0xffffffffu, sl, o);
            two_sum(s, os, s, e);
            sl = (sl + ol) + e;
        }
        two_sum(s * (1.0f / D), eps, s, e);
        sl = fmaf(sl, 1.0f / D, e);
        // 1 / sqrt(s + sl) = r + rl: r + r (1 - (s + sl) r^2) / 2
        const float r = rsqrtf(s), q = s * r, ql = fmaf(s, r, -q);
        float rl = 0.5f * r * fmaf(-sl * r, r, fmaf(-ql, r, fmaf(-q, r, 1.0f)));
        if (!(s < INFINITY)) rl = 0.0f;
        const F2 r2 = pair(r, r), rl2 = pair(rl, rl);
        F2 wv[4];
        {
            F2 t[2];
            load_w(w + ch_a, t);
            wv[0] = t[0], wv[1] = t[1];
            load_w(w + ch_b, t);
            wv[2] = t[0], wv[3] = t[1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            F2 n, nl;
            two_product(v[i], r2, n, nl);
            nl = ptx::fma2(v[i], rl2, nl);
            two_product(n, wv[i], v[i], lo[i]);
            lo[i] = ptx::fma2(nl, wv[i], lo[i]);
        }
    }
    if (!turned) return;
    // a b + c d, with al and cl behind a and c
    auto turn = [](F2 a, F2 al, F2 b, F2 c, F2 cl, F2 d, F2 &v, F2 &lo) {
        F2 p, pl, q, ql, e;
        two_product(a, b, p, pl);
        two_product(c, d, q, ql);
        two_sum(p, q, v, e);
        lo = ptx::fma2(al, b, ptx::fma2(cl, d, add2(add2(pl, ql), e)));
    };
    if (PAIRS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 x = v[i], xl = lo[i];
            turn(x, xl, cs[PAIRS ? i : 0], swapped(x), swapped(xl), sn[PAIRS ? i : 0], v[i], lo[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const F2 x = v[i], xl = lo[i], y = v[2 + i], yl = lo[2 + i];
            turn(x, xl, cs[i], y, yl, sn[i] ^ 0x8000000080000000ull, v[i], lo[i]);
            turn(y, yl, cs[i], x, xl, sn[i], v[2 + i], lo[2 + i]);
        }
    }
}

// v + lo towards zero, the last bit set where that is not exact: on the same side of every border.
__device__ __forceinline__ float to_odd(float v, float lo) {
    const float t = __fadd_rz(v, lo);
    return __uint_as_float(__float_as_uint(t) | (lo - (t - v) != 0.0f));
}

// U heads of a thread's own at a time.  D: channels of a head.  PAIRS: neighbours
// are a pair, else channels R / 2 apart.  CACHE: keys and values to the cache.
template <int D, bool PAIRS, int U, bool CACHE>
__global__ void __launch_bounds__(kRopeThreads, 4) qk_rope_kernel(const RopeArgs a) {
    constexpr int N8 = D / 8, kHeads = 32 / N8;   // lanes of a head, heads of a warp at a time
    static_assert(kRopeThreads >= 2 * D, "a thread to a weight");
    __shared__ __align__(16) float s_w[2][D];
    const int lane = threadIdx.x & 31, c = lane % N8, g = lane / N8;
    const int64_t job = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = job / a.parts;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    // Rounds of kHeads heads: of keys into the cache (the longest), of values, then of queries (and
    // of keys where there is no cache)
    const int heads = CACHE ? a.Hq : a.Hq + a.Hk;
    const int k_rounds = CACHE ? (a.Hk + kHeads - 1) / kHeads : 0, rounds = 2 * k_rounds + (heads + kHeads - 1) / kHeads;
    // This lane's channels: two fours, of which the second is the first one's partner
    // where pairs are half a rotation apart (no shuffles); of values eight neighbours.
    const bool turned = c < a.R / 8, split = !PAIRS && turned;
    const int ch_a = split ? 4 * c : 8 * c, ch_b = split ? a.R / 2 + 4 * c : 8 * c + 4;
    const bool there = t < a.T;
    const uint16_t *row = a.qkv + (there ? t * a.stride : 0);
    const int first = (int)(job - t * a.parts) * U, step = a.parts * U;
    uint2 raw[U][2];
    const uint16_t *from_a = row + g * D + ch_a, *from_b = row + g * D + ch_b;
    auto load = [&](int round) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int rd = round + u, h0 = (rd - 2 * k_rounds) * kHeads;
            raw[u][0] = raw[u][1] = make_uint2(0, 0);
            if (!CACHE || h0 >= 0) {
                if (h0 + g < heads) raw[u][0] = load_once(from_a + h0 * D), raw[u][1] = load_once(from_b + h0 * D);
            } else {
                const bool keys = rd < k_rounds;
                const int h = (rd - (keys ? 0 : k_rounds)) * kHeads + g;
                if (h < a.Hk) {
                    const uint16_t *p = row + (int64_t)(a.Hq + (keys ? 0 : a.Hk) + h) * D;
                    raw[u][0] = load_once(p + (keys ? ch_a : 8 * c));
                    raw[u][1] = load_once(p + (keys ? ch_b : 8 * c + 4));
                }
            }
        }
    };
    if (there) load(first);   // before what the position is waited for
    // the norms' weights, where registers would not hold them
    if (a.w_q || a.w_k) {
        const int i = threadIdx.x % D, k = threadIdx.x / D;
        const void *w = k ? a.w_k : a.w_q;
        if (k < 2 && w)
            s_w[k][i] = a.w_f32 ? static_cast<const float *>(w)[i]
                                : __uint_as_float((uint32_t)static_cast<const uint16_t *>(w)[i] << 16);
        __syncthreads();
    }
    if (!there) return;
    const int pos = a.R ? a.positions[t] : 0;
    const int slot = CACHE ? a.slots[t] : -1;
    if (pos < 0 || (a.R && pos >= a.max_positions) || slot < -1 || slot >= a.slots_in_cache) {
        if (lane == 0 && a.status) atomicOr(a.status, MOE_DEV_BAD_INDEX);
        return;   // the warp
    }
    // The angles: halves, of this lane's four pairs; neighbours, of each four's two pairs,
    // both cosines and (-sin, sin) twice
    F2 cs[PAIRS ? 4 : 2], sn[PAIRS ? 4 : 2];
    if (turned) {
        const float *table = a.cos_sin + (int64_t)pos * a.R + 4 * c;
        const uint4 x = *reinterpret_cast<const uint4 *>(table), y = *reinterpret_cast<const uint4 *>(table + a.R / 2);
        if (PAIRS) {
            const uint32_t neg = 0x80000000u;
            cs[0] = ptx::pack2(x.x, x.x), cs[1] = ptx::pack2(x.y, x.y);
            cs[PAIRS ? 2 : 0] = ptx::pack2(x.z, x.z), cs[PAIRS ? 3 : 1] = ptx::pack2(x.w, x.w);
            sn[0] = ptx::pack2(y.x ^ neg, y.x), sn[1] = ptx::pack2(y.y ^ neg, y.y);
            sn[PAIRS ? 2 : 0] = ptx::pack2(y.z ^ neg, y.z), sn[PAIRS ? 3 : 1] = ptx::pack2(y.w ^ neg, y.w);
        } else {
            cs[0] = ptx::pack2(x.x, x.y), cs[1] = ptx::pack2(x.z, x.w);
            sn[0] = ptx::pack2(y.x, y.y), sn[1] = ptx::pack2(y.z, y.w);
        }
    }
    const int64_t at = CACHE ? (((int64_t)(slot >> a.page_shift) * 2 * a.Hk) << a.page_shift) +
                                     (slot & ((1 << a.page_shift) - 1))
                               : 0;
    uint16_t *const q_row = a.q_out + (t * a.Hq + g) * D;
    // A head of this lane's, a query (or a key), to bf16; queries: whether all of the warp's are
    auto to_bf16 = [&](int h0, const uint2 (&now)[2], auto queries) {
        constexpr bool kQ = decltype(queries)::value;
        const int h = h0 + g;
        F2 x[2], y[2];
        unpack4(now[0], x);
        unpack4(now[1], y);
        if (a.w_q || (!kQ && a.w_k)) {
            F2 s2 = mul2(x[0], x[0]);
            s2 = ptx::fma2(x[1], x[1], s2);
            s2 = ptx::fma2(y[0], y[0], s2);
            s2 = ptx::fma2(y[1], y[1], s2);
            float sum = lo2(s2) + hi2(s2);
#pragma unroll
            for (int o = N8 / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = rsqrtf(sum * (1.0f / D) + a.eps);
            const F2 i2 = pair(inv, inv);
            const bool of_q = kQ || h < a.Hq;
            if (of_q ? a.w_q : a.w_k) {
                F2 w[2][2];
                load_w(s_w[of_q ? 0 : 1] + ch_a, w[0]), load_w(s_w[of_q ? 0 : 1] + ch_b, w[1]);
#pragma unroll
                for (int j = 0; j < 2; ++j) x[j] = mul2(mul2(x[j], i2), w[0][j]), y[j] = mul2(mul2(y[j], i2), w[1][j]);
            }
        }
        if (turned) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (PAIRS) {
                    x[j] = ptx::fma2(x[j], cs[j], mul2(pair(hi2(x[j]), lo2(x[j])), sn[j]));
                    y[j] = ptx::fma2(y[j], cs[PAIRS ? 2 + j : 0], mul2(pair(hi2(y[j]), lo2(y[j])), sn[PAIRS ? 2 + j : 0]));
                } else {
                    const F2 m = mul2(y[j], sn[j]);
                    y[j] = ptx::fma2(y[j], cs[j], mul2(x[j], sn[j]));
                    x[j] = ptx::fma2(x[j], cs[j], m ^ 0x8000000080000000ull);
                }
            }
        }
        uint16_t *const dst = kQ || h < a.Hq ? q_row + h0 * D : a.k_out + (t * a.Hk + h - a.Hq) * D;
        if (kQ || h < heads) store4(dst + ch_a, x), store4(dst + ch_b, y);
    };
    // Head h of the cache's (below 0: none), keys' heads before values': eight channels of this lane's
    // from 8 c on, or four and four
    auto encode8 = [&](const float (&v)[8], int h) {
        uint32_t m = 0;   // the largest magnitude
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));   // a block is four lanes
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t byte = mx4_scale_byte(m), mine = __shfl_sync(0xffffffffu, byte, (lane & ~(N8 - 1)) + (4 * c & (N8 - 1)));
        if (h < 0 || slot < 0) return;
        const int64_t r = at + ((int64_t)h << a.page_shift);
        reinterpret_cast<uint32_t *>(a.codes)[r * N8 + c] = mx4_codes8(v, byte);
        if (c < D / 32) a.scales[r * (D / 32) + c] = (uint8_t)mine;
    };
    auto encode44 = [&](const float (&v)[8], int h) {
        const float fa[8] = {v[0], v[1], v[2], v[3], 0.0f, 0.0f, 0.0f, 0.0f};
        const float fb[8] = {v[4], v[5], v[6], v[7], 0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t ma = 0, mb = 0, byte_a = 0, byte_b = 0, mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ma = max(ma, __float_as_uint(v[i]) & 0x7fffffffu);
            mb = max(mb, __float_as_uint(v[4 + i]) & 0x7fffffffu);
        }
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            uint32_t m = max(ch_a >> 5 == b ? ma : 0u, ch_b >> 5 == b ? mb : 0u);
#pragma unroll
            for (int o = N8 / 2; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const uint32_t byte = mx4_scale_byte(m);
            if (ch_a >> 5 == b) byte_a = byte;
            if (ch_b >> 5 == b) byte_b = byte;
            if (c == b) mine = byte;
        }
        if (h < 0 || slot < 0) return;
        const int64_t r = at + ((int64_t)h << a.page_shift);
        a.codes[r * (D / 4) + (ch_a >> 2)] = (uint16_t)mx4_codes8(fa, byte_a);
        a.codes[r * (D / 4) + (ch_b >> 2)] = (uint16_t)mx4_codes8(fb, byte_b);
        if (c < D / 32) a.scales[r * (D / 32) + c] = (uint8_t)mine;
    };
    // every thread of a warp goes through the same rounds: shuffles inside
    for (int round = first; round < rounds; round += step) {
        uint2 now[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u][0] = raw[u][0], now[u][1] = raw[u][1];
        load(round + step);
        const int q0 = (round - 2 * k_rounds) * kHeads;
        if (q0 >= 0 && q0 + U * kHeads <= a.Hq) {
#pragma unroll
            for (int u = 0; u < U; ++u) to_bf16(q0 + u * kHeads, now[u], std::true_type());
            continue;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int rd = round + u;
            if (rd >= rounds) break;   // the warp
            if (!CACHE || rd >= 2 * k_rounds) {
                to_bf16(q0 + u * kHeads, now[u], std::false_type());
            } else {
                const bool keys = rd < k_rounds;
                const int h = (rd - (keys ? 0 : k_rounds)) * kHeads + g;
                F2 x[2], v[4];
                unpack4(now[u][0], x), v[0] = x[0], v[1] = x[1];
                unpack4(now[u][1], x), v[2] = x[0], v[3] = x[1];
                float f[8];
                if (keys) {
                    F2 lo[4];
                    key_values<D, PAIRS>(v, lo, a.w_k ? s_w[1] : nullptr, ch_a, ch_b, a.eps, turned, cs, sn);
                    if (a.k_out && h < a.Hk) {
                        uint16_t *const dst = a.k_out + (t * a.Hk + h) * D;
                        store4(dst + ch_a, {v[0], v[1]}), store4(dst + ch_b, {v[2], v[3]});
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[2 * i] = to_odd(lo2(v[i]), lo2(lo[i]));
                        f[2 * i + 1] = to_odd(hi2(v[i]), hi2(lo[i]));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[2 * i] = lo2(v[i]), f[2 * i + 1] = hi2(v[i]);
                }
                const int head = h >= a.Hk ? -1 : keys ? h : a.Hk + h;
                if (PAIRS || !keys) encode8(f, head);
                else encode44(f, head);
            }
        }
    }
}

}  // namespace

int launch_qk_norm_rope(const moe_qk_rope *d, int T, const void *qkv, const int32_t *positions,
                        const float *cos_sin, const void *w_q, const void *w_k, void *q_out,
                        void *k_out, const moe_cache4 *cache, const int32_t *slots, int32_t *status,
                        cudaStream_t s) {
    RopeArgs a;
    a.qkv = static_cast<const uint16_t *>(qkv);
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.w_q = w_q;
    a.w_k = w_k;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.k_out = static_cast<uint16_t *>(k_out);
    a.codes = cache ? static_cast<uint16_t *>(cache->codes) : nullptr;
    a.scales = cache ? static_cast<uint8_t *>(cache->scales) : nullptr;
    a.slots = slots;
    a.status = status;
    a.stride = d->qkv_stride;
    a.slots_in_cache = cache ? (int64_t)cache->pages * cache->page : 0;
    a.Hq = d->q_heads;
    a.Hk = d->kv_heads;
    a.R = d->rope_dim;
    a.w_f32 = d->param_dtype == MOE_OUT_F32;
    a.max_positions = d->max_positions;
    a.page_shift = 0;
    if (cache)
        while ((1 << a.page_shift) < cache->page) ++a.page_shift;
    a.eps = d->eps;
    const bool pairs = d->style == MOE_ROPE_PAIRS;
    a.T = T;
    // Warps to a row: what takes the least time where each wave of the warps that run at once takes
    // 2.5 rounds to begin and end.  (5001 rows of 40 heads of 64: 19.0, 16.8, 17.6 and 25 us with 1,
    // 2, 3 and 10; 1000 rows: 8.2, 6.4, 5.8, 4.8, 5.9 and 6.5 with 1, 2, 3, 4, 5 and 10.)  Two heads of a
    // lane's at a time where there are many rounds and waves (8192 rows of 80 heads of 128: 60 us for
    // 68), one elsewhere (5001 rows: 16.8 for 20.3; 2048 rows of 80 heads of 128: 24.2 for 26.4).
    const int at_once = 32 / (d->dim / 8);
    const int most = (int)(cache ? ceil_div(a.Hq, at_once) + 2 * ceil_div(a.Hk, at_once) : ceil_div(a.Hq + a.Hk, at_once));
    const int64_t warps = (int64_t)sm_count() * 32;
    int64_t least = INT64_MAX;
    for (int p = 1; p <= std::min(most, 256); ++p) {
        const int64_t time = ceil_div((int64_t)T * p, warps) * (2 * ceil_div(most, p) + 5);
        if (time < least) least = time, a.parts = p;
    }
    const bool one = T <= warps || ceil_div(most, a.parts) < 12;
    auto go = [&](auto kern) {
        return launch_dependent(kern, dim3((unsigned)ceil_div((int64_t)T * a.parts, kRopeThreads / 32)), dim3(kRopeThreads), 0, s,
                                (const RopeArgs)a);
    };
    auto pick = [&](auto dim, auto p) {
        constexpr int D = decltype(dim)::value;
        constexpr bool P = decltype(p)::value;
        if (cache) return one ? go(qk_rope_kernel<D, P, 1, true>) : go(qk_rope_kernel<D, P, 2, true>);
        return one ? go(qk_rope_kernel<D, P, 1, false>) : go(qk_rope_kernel<D, P, 2, false>);
    };
    using std::integral_constant;
    if (d->dim == 64)
        return pairs ? pick(integral_constant<int, 64>(), std::true_type()) : pick(integral_constant<int, 64>(), std::false_type());
    return pairs ? pick(integral_constant<int, 128>(), std::true_type()) : pick(integral_constant<int, 128>(), std::false_type());
}

}  // namespace moe
