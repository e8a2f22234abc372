// Expert selection of one token by one warp, shared by the routing kernel and
// the few-token layer (the same ids and weights, bit for bit).
#pragma once

#include <cfloat>
#include <climits>
#include <stdint.h>

#include "../../include/moe_gb300.h"
#include "numerics.cuh"

namespace moe {

struct SelectArgs {
    int T, E, k, groups, topk_groups, topn, sigmoid, norm;
    float scaling;
    const float *logits, *bias;
    const int32_t *log2phys;
    int32_t *ids;
    float *w;
    int32_t *status;
    // optional: the FP8 quantisation of x (xq e4m3 [T, H], xs [T, H/128])
    const uint16_t *x;
    uint8_t *xq;
    float *xs;
    int H;
};

// warp-wide arg-max with ties to the lower index; every lane gets the result
__device__ __forceinline__ void warp_argmax(float &v, int &i) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, v, o);
        const int oi = __shfl_xor_sync(0xffffffffu, i, o);
        if (ov > v || (ov == v && oi < i)) {
            v = ov;
            i = oi;
        }
    }
}

// Scores of expert e of a token with logit lv: the score s (sigmoid) or the
// logit itself, and the value the selection compares.
__device__ __forceinline__ void expert_scores(const SelectArgs &a, int e, bool ok, float lv,
                                              float &sv, float &selv) {
    sv = lv;
    selv = lv;
    if (a.sigmoid) {
        sv = sigmoid_score(lv);
        selv = (ok && a.bias) ? __fadd_rn(sv, a.bias[e]) : sv;
    }
}

// Selection of token t from its experts' logits, scores and selection values
// (PL * 32 each, in shared memory): warp-wide, expert e = q*32 + lane in lane
// registers.  Writes row t of a.ids and a.w.
template <int PL>
__device__ __forceinline__ void warp_select(const SelectArgs &a, int t, int lane,
                                            const float *sh_l, const float *sh_s,
                                            const float *sh_sel) {
    float l[PL], s[PL], sel[PL];
    uint32_t valid = 0;
#pragma unroll
    for (int q = 0; q < PL; ++q) {
        const int e = q * 32 + lane;
        l[q] = sh_l[e];
        s[q] = sh_s[e];
        sel[q] = sh_sel[e];
        if (e < a.E) valid |= 1u << q;
    }
    uint32_t allowed = valid;

    if (a.groups > 1) {
        const int gs = a.E / a.groups;
        uint32_t gmask = 0;
        if (gs == 32 && a.topn <= 4) {
            // Groups of 32: lane L holds expert L of every group (group g is
            // q == g), so all groups reduce at once; same order, ties and
            // sums as the general path below.
            float gsum[PL];
            uint32_t taken = 0;
            for (int r = 0; r < a.topn; ++r) {
                float v[PL];
                int id[PL];
#pragma unroll
                for (int q = 0; q < PL; ++q) {
                    const bool ok = ((valid >> q) & 1u) && !((taken >> q) & 1u);
                    v[q] = ok ? sel[q] : -FLT_MAX;
                    id[q] = ok ? q * 32 + lane : INT_MAX;
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) {
#pragma unroll
                    for (int q = 0; q < PL; ++q) {
                        const float ov = __shfl_xor_sync(0xffffffffu, v[q], o);
                        const int oi = __shfl_xor_sync(0xffffffffu, id[q], o);
                        if (ov > v[q] || (ov == v[q] && oi < id[q])) {
                            v[q] = ov;
                            id[q] = oi;
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < PL; ++q) {
                    if (id[q] != INT_MAX && (id[q] & 31) == lane) taken |= 1u << q;
                    gsum[q] = (r == 0) ? v[q] : __fadd_rn(gsum[q], v[q]);
                }
            }
            for (int r = 0; r < a.topk_groups; ++r) {   // group scores are warp-uniform
                float bv = -FLT_MAX;
                int bg = INT_MAX;
#pragma unroll
                for (int q = 0; q < PL; ++q)
                    if (q < a.groups && !((gmask >> q) & 1u) &&
                        (gsum[q] > bv || (gsum[q] == bv && q < bg))) {
                        bv = gsum[q];
                        bg = q;
                    }
                if (bg != INT_MAX) gmask |= 1u << bg;
            }
        } else {
            float my_gscore = -FLT_MAX;
            for (int g = 0; g < a.groups; ++g) {
                uint32_t taken = 0;
                float sum = 0.0f;
                for (int r = 0; r < a.topn; ++r) {
                    float bv = -FLT_MAX;
                    int bi = INT_MAX;
#pragma unroll
                    for (int q = 0; q < PL; ++q) {
                        const int e = q * 32 + lane;
                        if (((valid >> q) & 1u) && !((taken >> q) & 1u) && e >= g * gs &&
                            e < (g + 1) * gs && (sel[q] > bv || (sel[q] == bv && e < bi))) {
                            bv = sel[q];
                            bi = e;
                        }
                    }
                    warp_argmax(bv, bi);
                    if (bi != INT_MAX && (bi & 31) == lane) taken |= 1u << (bi >> 5);
                    sum = (r == 0) ? bv : __fadd_rn(sum, bv);
                }
                if (lane == g) my_gscore = sum;
            }
            for (int r = 0; r < a.topk_groups; ++r) {
                float v = (lane < a.groups && !((gmask >> lane) & 1u)) ? my_gscore : -FLT_MAX;
                int i = (lane < a.groups && !((gmask >> lane) & 1u)) ? lane : INT_MAX;
                warp_argmax(v, i);
                if (i != INT_MAX) gmask |= 1u << i;
            }
        }
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            const int e = q * 32 + lane;
            if (((valid >> q) & 1u) && !((gmask >> (e / gs)) & 1u)) allowed &= ~(1u << q);
        }
    }

    // top-k by repeated arg-max; lane j keeps slot j
    uint32_t chosen = 0;
    int my_id = 0;
    float my_score = 0.0f;   // sigmoid s or softmax logit of slot `lane`
    for (int j = 0; j < a.k; ++j) {
        float bv = -FLT_MAX;
        int bi = INT_MAX;
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            const int e = q * 32 + lane;
            if (((allowed >> q) & 1u) && !((chosen >> q) & 1u) &&
                (sel[q] > bv || (sel[q] == bv && e < bi))) {
                bv = sel[q];
                bi = e;
            }
        }
        warp_argmax(bv, bi);
        if (bi == INT_MAX) {   // fewer candidates than k (rejected on the host)
            if (lane == 0 && a.status) atomicOr(a.status, MOE_DEV_BAD_EXPERT_ID);
            return;
        }
        const int owner = bi & 31, oq = bi >> 5;
        float sv = 0.0f;
#pragma unroll
        for (int q = 0; q < PL; ++q)
            if (q == oq) sv = s[q];
        sv = __shfl_sync(0xffffffffu, sv, owner);
        if (lane == owner) chosen |= 1u << oq;
        if (lane == j) {
            my_id = bi;
            my_score = sv;
        }
    }

    float w = 0.0f;
    if (a.sigmoid) {
        float total = 0.0f;
        for (int j = 0; j < a.k; ++j) total = __fadd_rn(total, __shfl_sync(0xffffffffu, my_score, j));
        w = a.norm ? __fmul_rn(__fdiv_rn(my_score, total), a.scaling)
                   : __fmul_rn(my_score, a.scaling);
    } else {
        // The ids above depend on the logits alone; the weights are
        // exp(l - m) / sum exp(l' - m) with m the largest logit.  Each
        // exponential is taken in fp32 (expf, within 2 ulp) of the exact
        // difference: l - m rounded, plus its rounding error from a two-sum,
        // applied in fp64 as exp(d + e) = exp(d) (1 + e).  Sums, the quotient
        // and the scaling are fp64, so a weight lies within 5.4e-7 (relative)
        // of the fp64 definition while its exponential is a normal fp32
        // number (l - m > -87).  This GPU's fp64 rate is a small fraction of
        // its fp32 rate.
        float m = -FLT_MAX;
#pragma unroll
        for (int q = 0; q < PL; ++q)
            if ((valid >> q) & 1u) m = fmaxf(m, l[q]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        auto ex = [&](float lv) -> double {
            const float d = __fsub_rn(lv, m);
            const float bb = __fsub_rn(d, lv);
            const float e = __fadd_rn(__fsub_rn(lv, __fsub_rn(d, bb)), __fsub_rn(-m, bb));
            const double x = (double)expf(d);
            return fma(x, (double)e, x);
        };
        double denom = 0.0;
        if (a.norm) {
            for (int j = 0; j < a.k; ++j) denom += ex(__shfl_sync(0xffffffffu, my_score, j));
        } else {
            double part = 0.0;
#pragma unroll
            for (int q = 0; q < PL; ++q)
                if ((valid >> q) & 1u) part += ex(l[q]);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
            denom = part;
        }
        w = (float)(ex(my_score) / denom * (double)a.scaling);
    }

    if (lane < a.k) {
        int id = my_id;
        if (a.log2phys) {
            id = a.log2phys[my_id];
            if (id < 0 || id >= a.E) {
                if (a.status) atomicOr(a.status, MOE_DEV_BAD_EXPERT_ID);
                id = -1;
            }
        }
        a.ids[(size_t)t * a.k + lane] = id;
        a.w[(size_t)t * a.k + lane] = w;
    }
}

}  // namespace moe
