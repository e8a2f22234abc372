// Norm of queries and keys for each head, the rotation by the token's position,
// and the write of keys and values into the four-bit cache, in one pass.
//
//   n = v / sqrt(mean(v^2) + eps) w
//   a, b -> a cos - b sin, b cos + a sin      (the pairs of the first R channels)
//
// A head is dim / 8 neighbouring lanes of eight channels: the norm's sum and the
// block maxima of MXFP4 (32 channels, four lanes) are butterflies over them, and
// with pairs half a rotation apart the partner's channels are another lane's.
// Everything is fp32 until the one rounding of each output; keys go to four
// bits from fp32, not by way of bf16.
//
// Bound by memory: a row is read and written once.  A CTA keeps one token's
// angles in registers over all of the token's heads that it takes, whose loads
// are under way together.
#include <cuda_bf16.h>

#include <algorithm>

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
    uint32_t *codes;
    uint8_t *scales;
    const int32_t *slots;
    int32_t *status;
    int64_t stride, slots_in_cache;
    int Hq, Hk, R, w_f32, max_positions, page_shift;
    float eps;
};

__device__ __forceinline__ void unpack8(const uint4 q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void load_w(const void *w, int f32, int c, float (&v)[8]) {
    if (f32) {
        const float4 a = static_cast<const float4 *>(w)[2 * c], b = static_cast<const float4 *>(w)[2 * c + 1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        unpack8(static_cast<const uint4 *>(w)[c], v);
    }
}

// U heads of a thread's own at a time.  D: channels of a head.  PAIRS: neighbours
// are a pair, else channels R / 2 apart.
template <int D, bool PAIRS, int U>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const RopeArgs a) {
    constexpr int N8 = D / 8, kHeads = kRopeThreads / N8;   // lanes of a head, heads at a time
    const int c = threadIdx.x % N8, g = threadIdx.x / N8;
    const int lane = threadIdx.x & 31, base = lane & ~(N8 - 1);
    const int64_t t = blockIdx.x;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int heads = a.Hq + a.Hk + (a.codes ? a.Hk : 0);
    const uint4 *row = reinterpret_cast<const uint4 *>(a.qkv + t * a.stride) + c;
    const int pos = a.R ? a.positions[t] : 0;
    const int slot = a.codes ? a.slots[t] : -1;
    if (pos < 0 || (a.R && pos >= a.max_positions) || slot < -1 || slot >= a.slots_in_cache) {
        if (threadIdx.x == 0 && a.status) atomicOr(a.status, MOE_DEV_BAD_INDEX);
        return;   // the CTA
    }
    // this lane's angles; past the rotated channels cos 1, sin 0
    float cs[8], sn[8];
    const int half = a.R / 16;   // in lanes
    const bool turned = c < 2 * half;
    const int partner = base + (c < half ? c + half : c - half);
    if (turned) {
        const float *table = a.cos_sin + (int64_t)pos * a.R;
        if (PAIRS) {
            const float4 x = *reinterpret_cast<const float4 *>(table + 4 * c);
            const float4 y = *reinterpret_cast<const float4 *>(table + a.R / 2 + 4 * c);
            cs[0] = cs[1] = x.x, cs[2] = cs[3] = x.y, cs[4] = cs[5] = x.z, cs[6] = cs[7] = x.w;
            sn[0] = sn[1] = y.x, sn[2] = sn[3] = y.y, sn[4] = sn[5] = y.z, sn[6] = sn[7] = y.w;
        } else {
            const int i = 8 * (c < half ? c : c - half);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 x = *reinterpret_cast<const float4 *>(table + i + 4 * j);
                const float4 y = *reinterpret_cast<const float4 *>(table + a.R / 2 + i + 4 * j);
                cs[4 * j] = x.x, cs[4 * j + 1] = x.y, cs[4 * j + 2] = x.z, cs[4 * j + 3] = x.w;
                sn[4 * j] = y.x, sn[4 * j + 1] = y.y, sn[4 * j + 2] = y.z, sn[4 * j + 3] = y.w;
            }
            if (c < half)
#pragma unroll
                for (int j = 0; j < 8; ++j) sn[j] = -sn[j];   // a cos - b sin; b cos + a sin
        }
    }
    const int64_t at = a.codes ? (((int64_t)(slot >> a.page_shift) * 2 * a.Hk) << a.page_shift) +
                                     (slot & ((1 << a.page_shift) - 1))
                               : 0;
    // every thread of a warp goes through the same rounds: shuffles inside
    for (int h0 = blockIdx.y * kHeads * U; h0 < heads; h0 += gridDim.y * kHeads * U) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * kHeads + g;
            if (h < heads) raw[u] = ptx::load_past_l1(row + (int64_t)h * N8);
            else raw[u] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * kHeads + g;
            if (h0 + u * kHeads >= heads) break;   // the CTA
            const bool is_v = h >= a.Hq + a.Hk, is_k = !is_v && h >= a.Hq;
            float v[8];
            unpack8(raw[u], v);
            const void *w = is_k ? a.w_k : a.w_q;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(v[j], v[j], sum);
#pragma unroll
            for (int o = N8 / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (w && !is_v) {
                const float inv = rsqrtf(sum * (1.0f / D) + a.eps);
                float wv[8];
                load_w(w, a.w_f32, c, wv);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = v[j] * inv * wv[j];
            }
            if (PAIRS) {
                if (turned && !is_v)
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const float x = v[j], y = v[j + 1];
                        v[j] = x * cs[j] - y * sn[j];
                        v[j + 1] = y * cs[j] + x * sn[j];
                    }
            } else if (a.R) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(0xffffffffu, v[j], turned ? partner : lane);
                if (turned && !is_v)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = fmaf(v[j], cs[j], o[j] * sn[j]);
            }
            if (h < a.Hq) {
                ptx::store_past_l1(reinterpret_cast<uint4 *>(a.q_out + (t * a.Hq + h) * D) + c, pack8(v));
            } else if (is_k && a.k_out) {
                ptx::store_past_l1(reinterpret_cast<uint4 *>(a.k_out + (t * a.Hk + h - a.Hq) * D) + c, pack8(v));
            }
            if (a.codes && h0 + (u + 1) * kHeads > a.Hq) {   // the CTA: some of these heads are cached
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                if (h >= a.Hq && h < heads && slot >= 0) {
                    const uint32_t byte = mx4_scale_byte(m);
                    // keys' heads, then values' heads, follow one another in a page
                    const int64_t r = at + ((int64_t)(h - a.Hq) << a.page_shift);
                    a.codes[r * N8 + c] = mx4_codes8(v, byte);
                    if ((c & 3) == 0) a.scales[(r * N8 + c) >> 2] = (uint8_t)byte;
                }
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
    a.codes = cache ? static_cast<uint32_t *>(cache->codes) : nullptr;
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
    auto go = [&](auto kern, int u) {
        const int at_once = kRopeThreads / (d->dim / 8) * u;
        const unsigned parts = (unsigned)std::min<int64_t>(ceil_div(heads, at_once), 65535);
        // few tokens: each round of heads in a CTA of its own
        const bool spread = (int64_t)T < 4 * sm_count();
        return launch_dependent(kern, dim3((unsigned)T, spread ? parts : 1u), dim3(kRopeThreads), 0, s,
                                (const RopeArgs)a);
    };
    const bool few = (int64_t)T * heads < 64 * sm_count();
    if (d->dim == 64) {
        if (pairs) return few ? go(qk_rope_kernel<64, true, 1>, 1) : go(qk_rope_kernel<64, true, 4>, 4);
        return few ? go(qk_rope_kernel<64, false, 1>, 1) : go(qk_rope_kernel<64, false, 4>, 4);
    }
    if (pairs) return few ? go(qk_rope_kernel<128, true, 1>, 1) : go(qk_rope_kernel<128, true, 4>, 4);
    return few ? go(qk_rope_kernel<128, false, 1>, 1) : go(qk_rope_kernel<128, false, 4>, 4);
}

}  // namespace moe
