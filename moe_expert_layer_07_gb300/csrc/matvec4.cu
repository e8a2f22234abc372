// Products of 1 to 16 rows with weights in four bits:
//   y[t, n] = sum_k x[t, k] W[n, k]
// x in bf16, W in MXFP4 or as integers with group scales and zero points.
//
// The least is reading W once, 4.25 bits a weight and more; what bounds it is the
// instructions around the products (150 to 350 a KB of W and warp) and, for
// few megabytes, the way in and out: a launch, x, the clusters' sums.  Measured
// with W of 30 to 40 MB, cold: MXFP4 10240 x 7168, one row 11.8 us (3.3 TB/s),
// 7168 x 8192 with 16 rows 15.7; integers in groups of 128, 7168 x 8192: one row
// 11.9, 16 rows 17.0 (1.8 TB/s); in groups of 32: 15.4 and 21.2.  MXFP4 of 65536 x 2048,
// where a cluster is not needed, one row 18.8 (3.8 TB/s).
//
// A warp takes 16 rows
// of W by slices of 128 of K, the M side of mma.sync m16n8k16, with 8 or 16
// rows of x as its N side.  Its slices of x stay in the warp's registers
// for all of its rows of W, so x costs nothing per weight: a CTA's warps share
// K among them, and where K is longer than a CTA's registers hold, the CTAs of a
// cluster do.  W comes by cp.async through a ring of each warp's own and leaves
// it by ldmatrix in the order of the products; the scales of a tile of rows
// come through the same ring, as the strips of four-byte words that hold them
// (their rows need not be aligned).
//
// Codes become fp16 unscaled (MXFP4: cvt; integers: 1024 + code or 1024 + 16 code
// put together from bits, minus the zero point, both exact), products of 32 of K
// are multiplied by the group's scale in fp32.  x is fp16 times a power of two for
// each row and warp (bf16 values have no more bits; off by up to 2^-29 of the
// largest among the warp's where they are as small).
//
// Sums: the K slices of a warp one after the other, then warps in order, then
// CTAs in order: the same bits each time.  Each CTA of a cluster pushes its sums to the
// one that adds them up (the pull it was before waited for the way there and back).
//
// Also measured, each against its time then: two CTAs to an SM with a slice to a warp 26.7 us for
// the first case's 12.6 (sums of 8 warps' slices twice as often); two tiles' code in line 18.3 for
// 16.9; integers taken bare as subnormal fp16 with the zero points off the sums 17.9 for 16.9.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "internal.h"
#include "mx4.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kMaxWarps = 16;
constexpr int kTileRows = 16, kSlice = 128;
constexpr int kItemBytes = kTileRows * kSlice / 2;
constexpr int kHold = 16;   // row tiles whose sums the CTAs of a cluster hold between exchanges
// Row tiles between two of a CTA's barriers, for 8 and 16 rows of x
__host__ __device__ constexpr int batch_tiles(int nq) { return 4 / nq; }
// Strips of scales and zero points: bytes of a row of W
constexpr int kScaleStrip = 32, kZeroStrip = 12;

constexpr int kStages = 4;   // what 16 warps' rings, of two slices each, leave room for
// Of the stages that are copied before the first products, those asked for before x is converted: with
// 3, 2, 1 and 0 int4 of 7168 x 8192 and 16 rows took 17.5, 16.9, 17.6 and 17.8 us, MXFP4 and one row 9.9,
// 9.8, 9.9 and 10.3 (copies and x come through the same queue).
constexpr int kBefore = 2;

// Kinds of weights: MXFP4, integers with one scale for a slice (groups of 128), with
// more than one (32, 64)
enum { kMx, kIntSlice, kIntBlocks };

// A stage of a warp's ring: a tile of 16 rows by the warp's slices, and its strips.
__host__ __device__ constexpr int stage_bytes(bool ints, int slices) {
    return slices * kItemBytes + kTileRows * (ints ? kScaleStrip + kZeroStrip : 12) + (ints ? 0 : 64 - 192 % 64) % 64;
}

struct MatvecArgs {
    const uint16_t *x;
    const uint8_t *w, *scales, *zeros;
    void *y;
    int T, N, K, slices, warps, per_cta, group_shift, s_f32, out_bf16;
    int t_shift;   // T <= 2^t_shift
    int scale_row, scale_words, zero_words;   // bytes of a row's scales; words of a strip
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ uint32_t fma_half2(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 h = __hfma2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b),
                              *reinterpret_cast<const __half2 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t add_half2(uint32_t a, uint32_t b) {
    const __half2 h = __hadd2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Eight integer codes less their zero point as fp16 pairs (0,4) (1,5) (2,6) (3,7), which x's
// fragments follow: 1024 + c - (1024 + z), and (1024 + 16 c) / 16 - (64 + z).
struct Zero {
    uint32_t one, sixteen;   // -(1024 + z), -(64 + z), twice each
    __device__ __forceinline__ Zero(uint32_t z4, int b) {   // byte b of four
        one = __byte_perm(z4, 0xe4u, 0x4040 + 0x101 * b);
        sixteen = __byte_perm(z4 << 4, 0xd4u, 0x4040 + 0x101 * b);
    }
};
// Constants that stay in registers: an instruction has room for one immediate.
struct IntBits {
    uint32_t lo, hi, k, sixteenth;
    __device__ __forceinline__ IntBits() {
        asm volatile("mov.b32 %0, 0x000f000f;\n\tmov.b32 %1, 0x00f000f0;\n\tmov.b32 %2, 0x64006400;\n\tmov.b32 %3, 0x2c002c00;"
                     : "=r"(lo), "=r"(hi), "=r"(k), "=r"(sixteenth));
    }
};
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ void widen_ints(uint32_t codes, const IntBits &k, const Zero &z, uint32_t (&h)[4]) {
    const uint32_t up = codes >> 8;
    h[0] = add_half2(and_or(codes, k.lo, k.k), z.one);
    h[1] = fma_half2(and_or(codes, k.hi, k.k), k.sixteenth, z.sixteen);
    h[2] = add_half2(and_or(up, k.lo, k.k), z.one);
    h[3] = fma_half2(and_or(up, k.hi, k.k), k.sixteenth, z.sixteen);
}

// The two halves of a barrier of the cluster; relaxed: one that orders no memory.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

__device__ __forceinline__ void write(const MatvecArgs &a, int t, int n, float v) {
    if (t >= a.T || n >= a.N) return;
    if (a.out_bf16) static_cast<__nv_bfloat16 *>(a.y)[(int64_t)t * a.N + n] = __float2bfloat16(v);
    else static_cast<float *>(a.y)[(int64_t)t * a.N + n] = v;
}

// NQ: rows of x in eights.  S: slices of a warp.
template <int KIND, int NQ, int S>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) matvec4_kernel(const MatvecArgs a) {
    constexpr bool INT = KIND != kMx;
    constexpr int kBatch = batch_tiles(NQ), kSums = NQ * 128;   // of a tile: [row of W][row of x]
    constexpr int kStage = stage_bytes(INT, S), kStrips = S * kItemBytes;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int rank = cluster_rank();
    const int ranks = a.slices > a.per_cta ? (a.slices + a.per_cta - 1) / a.per_cta : 1;
    const int cluster = blockIdx.x / ranks, clusters = gridDim.x / ranks;
    const int first_slice = rank * a.per_cta + warp * S, last_slice = min(a.slices, (rank + 1) * a.per_cta);
    const int tiles = (a.N + kTileRows - 1) / kTileRows;
    const int mine = cluster < tiles ? (tiles - cluster + clusters - 1) / clusters : 0;
    uint8_t *ring = smem + warp * kStages * kStage;
    const uint32_t ring_addr = smem_u32(ring);
    float *s_part = reinterpret_cast<float *>(smem + a.warps * kStages * kStage);   // [warps][kBatch][kSums]
    float *s_hold = s_part + a.warps * kBatch * kSums;                                // [ranks][hold_tiles][kSums]
    const int hold_tiles = (kHold + ranks - 1) / ranks, inv_ranks = 256 / ranks + 1;   // exact below kHold, to 8 ranks
    const uint32_t hold = smem_u32(s_hold);
    // MXFP4: [slice][row][block]
    float *s_scale = s_hold + (ranks > 1 ? ranks * hold_tiles * kSums : 0) + warp * (S * 64);
    const int row_bytes = a.K >> 1, groups = a.K >> a.group_shift;
    const int group0 = INT ? first_slice * (kSlice >> a.group_shift) : 0;
    const bool busy = first_slice < last_slice;
    // What this lane copies of a tile: pieces lane % 4 of rows lane / 4 and 8 more, and
    // words lane / 16, + 2 .. of the strips of row lane % 16, which begin anywhere in
    // their first word.
    const int row_a = lane >> 2, piece = lane & 3, row_s = lane & 15, word0 = lane >> 4;
    const uint32_t dst = ring_addr + row_a * 64 + ((piece ^ ((row_a >> 1) & 3)) << 4);
    const uint32_t dst_s = ring_addr + kStrips + row_s * (INT ? kScaleStrip : 12) + word0 * 4;
    const uint32_t dst_z = ring_addr + kStrips + kTileRows * kScaleStrip + row_s * kZeroStrip + word0 * 4;
    bool inside[S];
#pragma unroll
    for (int i = 0; i < S; ++i) inside[i] = busy && (first_slice + i) * 64 + piece * 16 < row_bytes;
    int n_next = cluster * kTileRows;   // the next tile to be copied
    const int64_t step_w = (int64_t)clusters * kTileRows * row_bytes, half_w = (int64_t)8 * row_bytes;
    const uint8_t *src = a.w + (int64_t)(n_next + row_a) * row_bytes + first_slice * 64 + piece * 16;
    // (Tiles are 16 rows apart and more: where a row's strip begins in its word is the same
    // for all of them.)
    const int64_t step_s = (int64_t)clusters * kTileRows * a.scale_row, step_z = (int64_t)clusters * kTileRows * groups;
    const int64_t at_s = (int64_t)(n_next + row_s) * a.scale_row + (INT ? group0 * (a.s_f32 ? 4 : 2) : first_slice * 4);
    const int64_t at_z = INT ? (int64_t)(n_next + row_s) * groups + group0 : 0;
    const uint8_t *src_s = a.scales + (at_s & ~(int64_t)3) + 4 * word0;
    const uint8_t *src_z = INT ? a.zeros + (at_z & ~(int64_t)3) + 4 * word0 : nullptr;
    const int words = INT ? a.scale_words : (a.K & 127) ? S + 1 : S;
    uint32_t to = 0, from = 0;   // stages of the ring
    // Copies the next tile into its stage of the ring
    auto fetch = [&]() {
        if (busy && n_next < a.N) {
            // all rows are there, and so many behind them that no strip's words pass the tensors' ends
            // (35 bytes of two a row, 11 of one)
            if (n_next + 3 * kTileRows <= a.N) {
#pragma unroll
                for (int i = 0; i < S; ++i)
                    if (inside[i]) {
                        cp_async16(dst + to + i * kItemBytes, src + i * 64);
                        cp_async16(dst + to + i * kItemBytes + 512, src + half_w + i * 64);
                    }
                if (word0 < words) cp_async4(dst_s + to, src_s, 4);
                if (KIND == kIntBlocks) {   // up to 9 words of scales, 3 of zero points
#pragma unroll
                    for (int word = 2; word < 10; word += 2)
                        if (word + word0 < words) cp_async4(dst_s + to + 4 * word, src_s + 4 * word, 4);
#pragma unroll
                    for (int word = 0; word < 4; word += 2)
                        if (word + word0 < a.zero_words) cp_async4(dst_z + to + 4 * word, src_z + 4 * word, 4);
                } else {                    // mostly one, and one
                    for (int word = 2; word < words; word += 2)
                        if (word + word0 < words) cp_async4(dst_s + to + 4 * word, src_s + 4 * word, 4);
                    if (INT)
                        for (int word = 0; word < a.zero_words; word += 2)
                            if (word + word0 < a.zero_words) cp_async4(dst_z + to + 4 * word, src_z + 4 * word, 4);
                }
            } else {
                const bool lo = n_next + row_a < a.N, hi = n_next + row_a + 8 < a.N;
#pragma unroll 1
                for (int i = 0; i < S; ++i) {
                    const bool in = busy && (first_slice + i) * 64 + piece * 16 < row_bytes;
                    if (lo && in) cp_async16(dst + to + i * kItemBytes, src + i * 64);
                    if (hi && in) cp_async16(dst + to + i * kItemBytes + 512, src + half_w + i * 64);
                }
                if (n_next + row_s < a.N) {   // not past the tensors' ends
                    const uint8_t *end_s = a.scales + (int64_t)a.N * a.scale_row, *end_z = a.zeros + (int64_t)a.N * groups;
                    for (int word = 0; word + word0 < words; word += 2)
                        if (src_s + 4 * word < end_s)
                            cp_async4(dst_s + to + 4 * word, src_s + 4 * word, (int)min((int64_t)4, (int64_t)(end_s - src_s) - 4 * word));
                    if (INT)
                        for (int word = 0; word + word0 < a.zero_words; word += 2)
                            if (src_z + 4 * word < end_z)
                                cp_async4(dst_z + to + 4 * word, src_z + 4 * word, (int)min((int64_t)4, (int64_t)(end_z - src_z) - 4 * word));
                }
            }
            src += step_w;
            src_s += step_s;
            if (INT) src_z += step_z;
        }
        n_next += clusters * kTileRows;
        cp_async_commit();
        to = to == (kStages - 1) * kStage ? 0 : to + kStage;
    };
    constexpr int kZeros = kStrips + kTileRows * kScaleStrip;
    // Where row r's strips begin in a stage
    auto strip_of = [&](int r, int &scales, int &zeros) {
        const uint32_t at = (uint32_t)(cluster * kTileRows + r) * groups + group0;   // its low bits
        scales = kStrips + r * kScaleStrip + (int)(at * (a.s_f32 ? 4 : 2) & 3);
        zeros = kZeros + r * kZeroStrip + (int)(at & 3);
    };
    int strip_s[2], strip_z[2];   // of rows g and g + 8, or of the row whose groups this lane makes numbers of
    strip_of(KIND == kIntBlocks ? lane >> 1 : g, strip_s[0], strip_z[0]);
    strip_of(KIND == kIntBlocks ? lane >> 1 : g + 8, strip_s[1], strip_z[1]);
    auto group_scale = [&](const uint8_t *strip, int gi) {
        return a.s_f32 ? reinterpret_cast<const float *>(strip)[gi]
                       : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(strip)[gi] << 16);
    };
    const IntBits bits;
    if (ranks > 1) cluster_arrive_relaxed();
    pdl_launch_dependents();
    pdl_wait();
    uint32_t xf[S][8][NQ][2];   // slices, steps of 16, rows of x
    float down[NQ][2];          // what undoes the powers of two of rows 8 n + 2 c, + 1
    uint4 all[NQ][S][4];        // before W: its copies would be waited for in line
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int t = 8 * n + g, k = (first_slice + i) * kSlice + 32 * b + 8 * c;
                all[n][i][b] = make_uint4(0, 0, 0, 0);
                if (t < a.T && k < a.K && first_slice + i < last_slice)
                    all[n][i][b] = __ldg(reinterpret_cast<const uint4 *>(a.x + (int64_t)t * a.K + k));
            }
#pragma unroll
    for (int i = 0; i < kBefore; ++i) fetch();
    // Pieces behind N or K are never copied: their products are not used (rows) or
    // are with x of zero (columns; the ring's bits are finite numbers, and the scales
    // are taken as zero).
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const uint4 (&raw)[S][4] = all[n];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint4 v = raw[i][b];
                const uint32_t k = 0x7fff7fffu;   // magnitudes of bf16 pairs order like whole numbers
                m = __vimax3_s16x2(m, v.x & k, v.y & k);
                m = __vimax3_s16x2(m, v.z & k, v.w & k);
            }
        m = max(m & 0xffffu, m >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // 2^(127 - ex) puts the row's largest into [2^14, 2^15), or leaves a tiny row's exponents
        // as they are
        const int ex = min(max((int)(m >> 7), 29), 254) - 14;
        const float un = __uint_as_float((uint32_t)ex << 23);
        down[n][0] = __shfl_sync(0xffffffffu, un, 8 * c);
        down[n][1] = __shfl_sync(0xffffffffu, un, 8 * c + 4);
        // bf16 to fp16 times that in the bits: the exponent is lowered by ex - 15 (in bf16's
        // place, with both types' biases); what falls below fp16's smallest is zero, and what
        // falls among its subnormal numbers off by up to 2^-15
        const uint32_t lower = (uint32_t)((-(ex - 15) << 7) & 0xffff) * 0x10001u;
        auto bits_of = [&](uint32_t w) {
            return (__viaddmax_s16x2_relu(w & 0x7fff7fffu, lower, 0u) << 3) | (w & 0x80008000u);
        };
        auto put = [&](auto convert) {
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t h[4] = {convert(raw[i][b].x), convert(raw[i][b].y), convert(raw[i][b].z), convert(raw[i][b].w)};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        xf[i][2 * b + j / 2][n][j & 1] =
                            INT ? __byte_perm(h[j / 2], h[2 + j / 2], j & 1 ? 0x7632 : 0x5410) : h[j];
                }
        };
        if (!__any_sync(0xffffffffu, m >= 0x7f80u)) {
            put(bits_of);
        } else {   // an infinity or a NaN
            put([&](uint32_t w) {
                uint32_t h = bits_of(w);
                if ((w & 0x7f80u) == 0x7f80u) h |= 0x7c00u | (w & 0x7fu) << 3;
                if ((w & 0x7f800000u) == 0x7f800000u) h |= 0x7c000000u | (w & 0x7f0000u) << 3;
                return h;
            });
        }
    }
#pragma unroll
    for (int i = kBefore; i < kStages - 1; ++i) fetch();
    const int mrow = (lane & 7) + ((lane >> 3) & 1) * 8, mblk = lane >> 4;

    // (Not unrolled: with two tiles' code in line, the instruction cache was what 16 rows of x
    // waited for.)
#pragma unroll 1
    for (int it = 0; it < mine; ++it) {
        const int slot_in_batch = it % kBatch;
        float acc[NQ][4];
        cp_async_wait<kStages - 2>();
        __syncwarp();
        fetch();
        uint8_t *stage = ring + from;
        const uint32_t slot = ring_addr + from;
        from = from == (kStages - 1) * kStage ? 0 : from + kStage;
        const int n0 = (cluster + it * clusters) * kTileRows;
        if (KIND == kMx) {
            // Scales as numbers, each formed once: lane (row, half) two blocks of each slice.
            // 2^(byte - 127); byte 0 (2^-127) counts as zero, 255 as infinity: its codes are
            // zero, and zero times it NaN.
            const int row = lane >> 1, half = lane & 1;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const uint32_t *strip = reinterpret_cast<const uint32_t *>(stage + kStrips + row * 12) + i;
                uint32_t w = strip[0];
                if (a.K & 127) {
                    w = __funnelshift_r(w, strip[1], 8 * (((n0 + row) * (a.K >> 5)) & 3));   // 4 first_slice: no matter
                    if ((first_slice + i) * 4 + 4 > a.K >> 5)   // blocks behind K
                        w &= (1u << 8 * max(0, (a.K >> 5) - (first_slice + i) * 4)) - 1u;
                }
                if (first_slice + i >= last_slice) w = 0;
                w >>= 16 * half;
                *reinterpret_cast<float2 *>(s_scale + i * 64 + row * 4 + 2 * half) =
                    make_float2(__uint_as_float((w & 0xffu) << 23), __uint_as_float((w >> 8 & 0xffu) << 23));
            }
            __syncwarp();
        }
        if (KIND == kIntBlocks) {
            // The same for integers, into the strips' places: scales as fp32, zero points as bytes.
            // (For the one group of a slice it took as long as forming them where they are used.)
            const int row = lane >> 1, half = lane & 1, per = kSlice >> a.group_shift;   // groups of a slice: 2 or 4
            float f[S][2];
            uint32_t z[S][2];
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int gi = i * per + (per == 4 ? 2 * half + x : half);
                    const bool there = group0 + gi < groups;
                    f[i][x] = there ? group_scale(stage + strip_s[0], gi) : 0.0f;
                    z[i][x] = a.zeros && there ? stage[strip_z[0] + gi] & 15u : 8u;
                }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < S; ++i) {
                *reinterpret_cast<float2 *>(stage + kStrips + row * kScaleStrip + 16 * i + 8 * half) = make_float2(f[i][0], f[i][1]);
                *reinterpret_cast<uint16_t *>(stage + kZeros + row * kZeroStrip + 4 * i + 2 * half) = (uint16_t)(z[i][0] | z[i][1] << 8);
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < S; ++i) {
            // scales (and zero points) of rows g and g + 8, for the four blocks of 32 or the slice
            constexpr int kB = KIND == kIntSlice ? 1 : 4;
            float sc[2][kB];
            uint32_t zp[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = g + 8 * r;
                if (KIND == kIntSlice) {
                    const bool there = group0 + i < groups;
                    sc[r][0] = there ? group_scale(stage + strip_s[r], i) : 0.0f;
                    zp[r] = a.zeros && there ? stage[strip_z[r] + i] & 15u : 8u;
                } else {
                    const float *fs = INT ? reinterpret_cast<const float *>(stage + kStrips + row * kScaleStrip) + 4 * i
                                          : s_scale + i * 64 + row * 4;
                    const float4 f = *reinterpret_cast<const float4 *>(fs);
                    sc[r][0] = f.x, sc[r][1 % kB] = f.y, sc[r][2 % kB] = f.z, sc[r][3 % kB] = f.w;
                    if (INT) zp[r] = *reinterpret_cast<const uint32_t *>(stage + kZeros + row * kZeroStrip + 4 * i);
                }
            }
            float d[NQ][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t w[4];
                ldm4(slot + i * kItemBytes + mrow * 64 + (((2 * x + mblk) ^ ((mrow >> 1) & 3)) << 4), w);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int b = 2 * x + y;
                    uint32_t w0[4], w1[4];
                    if (INT) {
                        widen_ints(w[2 * y], bits, Zero(zp[0], b % kB), w0);
                        widen_ints(w[2 * y + 1], bits, Zero(zp[1], b % kB), w1);
                    } else {
                        mx4_half8(w[2 * y], w0);
                        mx4_half8(w[2 * y + 1], w1);
                    }
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        // one sum for what shares a scale
                        if (b % (4 / kB) == 0) mma16816_first(d[n], w0[0], w1[0], w0[1], w1[1], xf[i][2 * b][n][0], xf[i][2 * b][n][1]);
                        else mma16816(d[n], w0[0], w1[0], w0[1], w1[1], xf[i][2 * b][n][0], xf[i][2 * b][n][1]);
                        mma16816(d[n], w0[2], w1[2], w0[3], w1[3], xf[i][2 * b + 1][n][0], xf[i][2 * b + 1][n][1]);
                        if (b % (4 / kB) == 4 / kB - 1) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                acc[n][j] = i + b < 4 / kB ? d[n][j] * sc[j >> 1][b % kB] : fmaf(d[n][j], sc[j >> 1][b % kB], acc[n][j]);
                        }
                    }
                }
            }
        }
        // the warps' sums of a batch of tiles
        if (slot_in_batch == 0 && it) __syncthreads();   // those of the batch before have been read
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float *p = s_part + (warp * kBatch + slot_in_batch) * kSums + 8 * n + 2 * c;
            *reinterpret_cast<float2 *>(p + g * 8 * NQ) = make_float2(acc[n][0] * down[n][0], acc[n][1] * down[n][1]);
            *reinterpret_cast<float2 *>(p + (g + 8) * 8 * NQ) = make_float2(acc[n][2] * down[n][0], acc[n][3] * down[n][1]);
        }
        if (slot_in_batch != kBatch - 1 && it != mine - 1) continue;
        const int batch = slot_in_batch + 1, it0 = it - slot_in_batch;
        __syncthreads();
        if (ranks > 1 && it0 % kHold == 0) cluster_wait();   // the other CTAs run, and have read what they held
        for (int i = tid; i < batch << (4 + a.t_shift); i += a.warps * 32) {
            const int t = i & ((1 << a.t_shift) - 1), row = i >> a.t_shift & 15, slot = i >> (4 + a.t_shift), j = row * 8 * NQ + t;
            const float *p = s_part + slot * kSums + j;
            float v = 0.0f;
#pragma unroll 4
            for (int q = 0; q < a.warps; ++q) v += p[q * kBatch * kSums];
            const int at = it0 + slot, held = at % kHold, share = held * inv_ranks >> 8;   // held / ranks
            if (ranks > 1)   // to the CTA that adds them up
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(
                                 hold + 4 * ((rank * hold_tiles + share) * kSums + j), held - share * ranks)), "f"(v) : "memory");
            else write(a, t, (cluster + at * clusters) * kTileRows + row, v);
        }
        static_assert(kHold % kBatch == 0, "a batch is held as a whole");
        if (ranks > 1 && (it % kHold == kHold - 1 || it == mine - 1)) {
            // the CTAs' sums together: CTA r finishes tiles r, r + ranks .. of what is held
            const int held = it % kHold + 1, base = it - it % kHold, own = (held - rank + ranks - 1) / ranks;
            cluster_sync();
            for (int i = tid; i < own << (4 + a.t_shift); i += a.warps * 32) {
                const int t = i & ((1 << a.t_shift) - 1), row = i >> a.t_shift & 15, slot = i >> (4 + a.t_shift);
                const float *p = s_hold + slot * kSums + row * 8 * NQ + t;
                float v = 0.0f;
                for (int r = 0; r < ranks; ++r) v += p[r * hold_tiles * kSums];
                write(a, t, (cluster + (base + rank + slot * ranks) * clusters) * kTileRows + row, v);
            }
            if (it != mine - 1) cluster_arrive();   // they may be overwritten
        }
    }
    cp_async_wait<0>();
}

// Clusters of c that run at a time on the current device: asked for once each kernel, size of a cluster
// and number of warps, which also say how much shared memory there is.
template <int KIND, int NQ, int S>
int clusters_at_once(const cudaLaunchConfig_t &c, int ranks, int warps) {
    static std::atomic<int> known[16][9][kMaxWarps + 1];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 1;
    std::atomic<int> *const place = dev < 16 ? &known[dev][ranks][warps] : nullptr;
    if (place && (n = place->load(std::memory_order_relaxed)) != 0) return n;
    if (cudaOccupancyMaxActiveClusters(&n, matvec4_kernel<KIND, NQ, S>, &c) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return 1;
    }
    if (place) place->store(n, std::memory_order_relaxed);
    return n;
}

template <int KIND, int NQ, int S>
int launch(const MatvecArgs &a, int ranks, cudaStream_t s) {
    const auto kern = matvec4_kernel<KIND, NQ, S>;
    const int hold = ranks > 1 ? ranks * (int)ceil_div(kHold, ranks) : 0;   // seven ranks: kHold + 5
    auto bytes = [](int warps, int hold) {
        return warps * kStages * stage_bytes(KIND != kMx, S) + (warps * batch_tiles(NQ) + hold) * NQ * 128 * 4 +
               (KIND == kMx ? warps * S * 64 * 4 : 0);
    };
    const int smem = bytes(a.warps, hold);
    // (the most that any call takes: calls of several threads set the same)
    MOE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(kMaxWarps, kHold + 5)));
    cudaLaunchConfig_t c = {};
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
    // All clusters at once.  Not every SM has neighbours for one of more than two: 36 of four run, 28
    // of five, 15 of seven or eight, and a second round of a few takes as long as the first.
    const int tiles = (int)ceil_div(a.N, kTileRows);
    int clusters = std::max(1, sm_count() / ranks);
    c.gridDim = dim3((unsigned)(ranks * clusters));
    if (ranks > 2) clusters = std::min(clusters, clusters_at_once<KIND, NQ, S>(c, ranks, a.warps));
    c.gridDim = dim3((unsigned)(ranks * std::min(tiles, clusters)));
    const cudaError_t e = cudaLaunchKernelEx(&c, kern, (const MatvecArgs)a);
    return e == cudaSuccess ? MOE_OK : cuda_fail("cudaLaunchKernelEx", e);
}

}  // namespace

int launch_w4_matvec(const moe_w4 *d, int T, const void *x, const void *codes, const void *scales,
                     const void *zeros, void *y, int out_dtype, cudaStream_t s) {
    MatvecArgs a;
    a.x = static_cast<const uint16_t *>(x);
    a.w = static_cast<const uint8_t *>(codes);
    a.scales = static_cast<const uint8_t *>(scales);
    a.zeros = static_cast<const uint8_t *>(zeros);
    a.y = y;
    a.T = T;
    for (a.t_shift = 0; 1 << a.t_shift < T; ++a.t_shift);
    a.N = d->n_out;
    a.K = d->k_dim;
    a.slices = (int)ceil_div(a.K, kSlice);
    a.group_shift = d->group == 32 ? 5 : d->group == 64 ? 6 : 7;
    a.s_f32 = d->scale_dtype == MOE_OUT_F32;
    a.out_bf16 = out_dtype == MOE_OUT_BF16;
    // Slices a warp and CTAs a cluster: x's registers are 16 (8 rows) or 32 a slice
    const int per_warp = a.slices > kMaxWarps ? 2 : 1;
    int ranks = 1;
    while (ranks * kMaxWarps * per_warp < a.slices) ++ranks;   // 32768 of K: 8
    a.warps = (int)ceil_div(ceil_div(a.slices, ranks), per_warp);
    a.per_cta = a.warps * per_warp;
    ranks = (int)ceil_div(a.slices, a.per_cta);
    const int groups = a.K / d->group, size = a.s_f32 ? 4 : 2, strip = per_warp * kSlice / d->group;   // a strip's groups
    a.scale_row = d->kind == MOE_W4_INT ? groups * size : groups;
    a.scale_words = a.s_f32 ? strip : (strip * 2 + 2 + 3) / 4;
    a.zero_words = zeros ? (strip + 3 + 3) / 4 : 0;
    const bool wide = T > 8;
    auto go = [&](auto kind) {
        constexpr int K = decltype(kind)::value;
        if (per_warp == 1) return wide ? launch<K, 2, 1>(a, ranks, s) : launch<K, 1, 1>(a, ranks, s);
        return wide ? launch<K, 2, 2>(a, ranks, s) : launch<K, 1, 2>(a, ranks, s);
    };
    if (d->kind == MOE_W4_MX) return go(std::integral_constant<int, kMx>());
    if (d->group == kSlice) return go(std::integral_constant<int, kIntSlice>());
    return go(std::integral_constant<int, kIntBlocks>());
}

}  // namespace moe
