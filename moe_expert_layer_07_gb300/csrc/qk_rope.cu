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
// bits from fp32, not by way of bf16.
//
// Bound by memory, and by the issue of instructions nearly as much (140 for two
// heads of 128 of a warp's before rounds of queries alone had code of their own):
// a row is read and written once.  A warp keeps one token's angles in registers over the
// heads that it takes, the next ones' loads under way.  8192 rows of 64 + 16 heads of 128:
// 54 us (5.65 TB/s), into the cache 70 (4.4); 5001 rows of 32 + 8 heads of 64 into the
// cache 16.3 us (2.9 TB/s: two waves of warps, 4 us of it launch and end); 7 rows 2.3
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
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

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
__device__ __forceinline__ uint32_t magnitude(const F2 (&v)[2]) {   // the largest of four
    const uint32_t k = 0x7fffffffu;
    return max(max((uint32_t)v[0] & k, (uint32_t)(v[0] >> 32) & k), max((uint32_t)v[1] & k, (uint32_t)(v[1] >> 32) & k));
}

// U heads of a thread's own at a time.  D: channels of a head.  PAIRS: neighbours
// are a pair, else channels R / 2 apart.
template <int D, bool PAIRS, int U>
__global__ void __launch_bounds__(kRopeThreads, 4) qk_rope_kernel(const RopeArgs a) {
    constexpr int N8 = D / 8, kHeads = 32 / N8;   // lanes of a head, heads of a warp at a time
    static_assert(kRopeThreads >= 2 * D, "a thread to a weight");
    __shared__ __align__(16) float s_w[2][D];
    const int lane = threadIdx.x & 31, c = lane % N8, g = lane / N8;
    const int64_t job = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = job / a.parts;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int heads = a.Hq + a.Hk + (a.codes ? a.Hk : 0), keyed = a.Hq + a.Hk;
    // This lane's channels: two fours, of which the second is the first one's partner
    // where pairs are half a rotation apart (no shuffles); of values eight neighbours.
    const bool turned = c < a.R / 8, split = !PAIRS && turned;
    const int ch_a = split ? 4 * c : 8 * c, ch_b = split ? a.R / 2 + 4 * c : 8 * c + 4;
    const bool there = t < a.T;
    const uint16_t *row = a.qkv + (there ? t * a.stride : 0);
    const int first = (int)(job - t * a.parts) * kHeads * U, step = a.parts * kHeads * U;
    uint2 raw[U][2];
    const uint16_t *from_a = row + g * D + ch_a, *from_b = row + g * D + ch_b;
    auto load = [&](int h0) {
        if (h0 + U * kHeads <= keyed) {   // no values
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw[u][0] = load_once(from_a + h0 * D + u * kHeads * D);
                raw[u][1] = load_once(from_b + h0 * D + u * kHeads * D);
            }
            return;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * kHeads + g;
            raw[u][0] = raw[u][1] = make_uint2(0, 0);
            if (h < heads) {
                const uint16_t *p = row + h * D;
                raw[u][0] = load_once(p + (h < keyed ? ch_a : 8 * c));
                raw[u][1] = load_once(p + (h < keyed ? ch_b : 8 * c + 4));
            }
        }
    };
    if (there) load(first);   // before what the position is waited for
    // the norms' weights, where registers would not hold them
    if (a.w_q || a.w_k) {
        const int i = threadIdx.x % D, k = threadIdx.x / D;
        const void *w = k ? a.w_k : a.w_q;
        if (k < 2 && w) s_w[k][i] = a.w_f32 ? static_cast<const float *>(w)[i] : __uint_as_float((uint32_t)static_cast<const uint16_t *>(w)[i] << 16);
        __syncthreads();
    }
    if (!there) return;
    const int pos = a.R ? a.positions[t] : 0;
    const int slot = a.codes ? a.slots[t] : -1;
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
    const int64_t at = a.codes ? (((int64_t)(slot >> a.page_shift) * 2 * a.Hk) << a.page_shift) +
                                     (slot & ((1 << a.page_shift) - 1))
                               : 0;
    uint16_t *const q_row = a.q_out + (t * a.Hq + g) * D;
    // U heads of this lane's; all of the warp's are queries, or any
    auto heads_of = [&](int h0, const uint2 (&now)[U][2], auto only_queries) {
        constexpr bool kQ = decltype(only_queries)::value;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * kHeads + g;
            if (!kQ && h0 + u * kHeads >= heads) break;   // the warp
            const bool is_v = !kQ && h >= keyed, is_k = !kQ && !is_v && h >= a.Hq;
            F2 x[2], y[2];
            unpack4(now[u][0], x);
            unpack4(now[u][1], y);
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
                if (!is_v && (of_q ? a.w_q : a.w_k)) {
                    F2 w[2][2];
                    load_w(s_w[of_q ? 0 : 1] + ch_a, w[0]), load_w(s_w[of_q ? 0 : 1] + ch_b, w[1]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[j] = mul2(mul2(x[j], i2), w[0][j]), y[j] = mul2(mul2(y[j], i2), w[1][j]);
                }
            }
            if (turned && !is_v) {
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
            if (kQ) {
                uint16_t *const dst = q_row + h0 * D + u * kHeads * D;
                store4(dst + ch_a, x), store4(dst + ch_b, y);
                continue;
            }
            uint16_t *dst = h < a.Hq ? q_row + (h0 + u * kHeads) * D : is_k && a.k_out ? a.k_out + (t * a.Hk + h - a.Hq) * D : nullptr;
            if (dst) store4(dst + ch_a, x), store4(dst + ch_b, y);
            if (a.codes && h0 + (u + 1) * kHeads > a.Hq) {   // the warp: some of these heads are cached
                // the blocks that this lane's channels are in, and their largest magnitudes
                const int at_a = is_v ? 8 * c : ch_a, at_b = is_v ? 8 * c + 4 : ch_b;
                const int blk_a = at_a >> 5, blk_b = at_b >> 5;
                const uint32_t ma = magnitude(x), mb = magnitude(y);
                uint32_t byte_a = 0, byte_b = 0, mine = 0;
#pragma unroll
                for (int b = 0; b < D / 32; ++b) {
                    uint32_t m = max(blk_a == b ? ma : 0u, blk_b == b ? mb : 0u);
#pragma unroll
                    for (int o = N8 / 2; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const uint32_t byte = mx4_scale_byte(m);
                    if (blk_a == b) byte_a = byte;
                    if (blk_b == b) byte_b = byte;
                    if (c == b) mine = byte;
                }
                if (h >= a.Hq && h < heads && slot >= 0) {
                    // keys' heads, then values' heads, follow one another in a page
                    const int64_t r = at + ((int64_t)(h - a.Hq) << a.page_shift);
                    const float fa[8] = {lo2(x[0]), hi2(x[0]), lo2(x[1]), hi2(x[1]), 0.0f, 0.0f, 0.0f, 0.0f};
                    const float fb[8] = {lo2(y[0]), hi2(y[0]), lo2(y[1]), hi2(y[1]), 0.0f, 0.0f, 0.0f, 0.0f};
                    a.codes[r * (D / 4) + (at_a >> 2)] = (uint16_t)mx4_codes8(fa, byte_a);
                    a.codes[r * (D / 4) + (at_b >> 2)] = (uint16_t)mx4_codes8(fb, byte_b);
                    if (c < D / 32) a.scales[r * (D / 32) + c] = (uint8_t)mine;
                }
            }
        }
    };
    // every thread of a warp goes through the same rounds: shuffles inside
    for (int h0 = first; h0 < heads; h0 += step) {
        uint2 now[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u][0] = raw[u][0], now[u][1] = raw[u][1];
        load(h0 + step);
        if (h0 + U * kHeads <= a.Hq) heads_of(h0, now, std::true_type());
        else heads_of(h0, now, std::false_type());
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
    const int heads = a.Hq + a.Hk + (cache ? a.Hk : 0);
    const bool pairs = d->style == MOE_ROPE_PAIRS;
    a.T = T;
    // Warps to a row: what takes the least time where each wave of the warps that run at once takes
    // 2.5 rounds to begin and end.  (5001 rows of 40 heads of 64: 19.0, 16.8, 17.6 and 25 us with 1,
    // 2, 3 and 10; 1000 rows: 8.2, 6.4, 5.8, 4.8, 5.9 and 6.5 with 1, 2, 3, 4, 5 and 10.)  Two heads of a
    // lane's at a time where there are many rounds and waves (8192 rows of 80 heads of 128: 60 us for
    // 68), one elsewhere (5001 rows: 16.8 for 20.3; 2048 rows of 80 heads of 128: 24.2 for 26.4).
    const int at_once = 32 / (d->dim / 8);
    const int most = (int)ceil_div(heads, at_once);
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
        return one ? go(qk_rope_kernel<D, P, 1>) : go(qk_rope_kernel<D, P, 2>);
    };
    using std::integral_constant;
    if (d->dim == 64)
        return pairs ? pick(integral_constant<int, 64>(), std::true_type()) : pick(integral_constant<int, 64>(), std::false_type());
    return pairs ? pick(integral_constant<int, 128>(), std::true_type()) : pick(integral_constant<int, 128>(), std::false_type());
}

}  // namespace moe
