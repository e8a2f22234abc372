// Attention of few query rows over the four-bit cache:
//   o = sum_j softmax_j(scale q . k_j) v_j
//
// One pass over the tokens with a running maximum m and sum l for each row:
//   s = scale log2(e) q . k,  p = 2^(s - m + 11),  l += p,  o += p v
// Rows are the query heads of one KV head, for one or more query tokens; 8, 16
// or 32 of them are the N side of the tensor cores' mma.sync m16n8k16, tokens
// (for S^T = K Q^T) and channels (for O^T = V^T P^T) the M side, so that a key
// or value is unpacked once for all rows and no row of a product is wasted when
// there are eight.  tcgen05 would need both operands in shared memory, 16 bits
// wide: 176 bytes a clock of an SM at the cache's full rate, where it has 128.
//
// Four-bit codes become fp16 with cvt (two an instruction).  The keys' scales are
// powers of two for 32 channels: they multiply the fp32 product of each block.
// Values are fp16 numbers where their scale is 2^-23 to 2^13: one more product for
// each pair of them.  (The scales times P instead, relative to the largest met, took less
// and lost what lay 22 binades below it, also below tokens that a row does not see.)
// A tile with other scales has them taken in bands of 37 binades, each with a
// product of its own.  m is raised only when a score passes it by 4 (in log2);
// then o is scaled.  q is fp16 times a power of two for each row: bf16
// values have no more bits, and what is 2^-38 of the row's largest is lost.
//
// A warp works alone: it copies tiles of 16 tokens (keys, values and scales, 2176
// bytes at 128 channels) into a ring of its own with cp.async and has its own m,
// l and o; ldmatrix gives both operands in the order of the products, the
// values transposed in units of four codes.  Shared memory holds 16-byte pieces
// exchanged within rows so that ldmatrix meets no bank twice.
//
// Work is cut into units of 128 tokens (eight warps) of a request, KV head and
// group of rows; a CTA takes as many neighbouring units as any other, whatever
// the requests' lengths.  A request that is cut between CTAs leaves partial
// results in the workspace (at most two a CTA), which a second kernel joins.
//
// Measured (cold): 48 requests of 64 to 16384 tokens, 64 query heads on 8 of 128, 61.1 us (3.7 TB/s
// of the cache; 58.4 with the scales times P); two of 131073 with three query tokens, 40 heads on 8, 94.5 (3.0
// TB/s; 97.6); one of 4097 tokens 11.1, two thirds of it launches, the way to the first tokens and the join.
// What bounds the large ones is the unpacking: 370 instructions a warp for 16 tokens
// of 128 channels, three quarters of what an SM can issue while it streams (one CTA of an SM
// is as fast alone as two are together), half of it on the integer pipe, which converts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "attention4.cuh"
#include "mx4.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kThreads = kAttnWarps * 32;
// What the beginning and end of a piece cost, in units: queries, the first tiles'
// way from memory, the warps' sums.  Measured with 3, 4, 5, 6 and 8 (the scales still times P): 48 requests of 64
// to 16384 tokens 63.9, 58.4, 58.7, 60.0 and 62.0 us.
constexpr int kPieceUnits = 4;
constexpr float kRest = 11.0f;     // where a raised maximum is put (log2)
// Scale bytes with which every value is an fp16 number; others lie in bands of so many.
constexpr int kLeastHalf = 104, kBand = 37;

// Mark of a value that is NaN.
constexpr uint32_t kNan = 0x8000u;

// Whether a row that sees a pair of tokens (seen: halves that are not zero) sees a value that is NaN.
__device__ __forceinline__ bool sees_nan(uint32_t seen, uint32_t scales) {
    return ((scales & 0xffffu) == kNan && (seen & 0xffffu)) || (scales >> 16 == kNan && seen >> 16);
}

// N words of shared memory, as bits or as floats.
__device__ __forceinline__ void put(uint32_t &v, uint32_t w) { v = w; }
__device__ __forceinline__ void put(float &v, uint32_t w) { v = __uint_as_float(w); }
template <int N, typename T>
__device__ __forceinline__ void load_blocks(T (&v)[N], const T *p) {
    if (N == 4) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        put(v[0], w.x), put(v[1], w.y), put(v[2 % N], w.z), put(v[3 % N], w.w);
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        put(v[0], w.x), put(v[1], w.y);
    }
}

// A word of eight codes, of channels 0 .. 3 for one token and for the next, in the
// order that gives pairs of tokens: channels 0, 2, 1, 3.
__device__ __forceinline__ uint32_t token_pairs(uint32_t w) {
    const uint32_t x = (w ^ (w >> 12)) & 0x0000f0f0u;
    return w ^ x ^ (x << 12);
}

template <int D, int NQ>
struct Shape {
    static constexpr int kBlocks = D / 32;              // channel blocks
    static constexpr int kRow = D / 2;                  // bytes of a token's codes
    static constexpr int kCodes = kAttnTile * kRow;     // of a tile's keys or values
    static constexpr int kScales = kAttnTile * kBlocks;
    static constexpr int kStage = 2 * (kCodes + kScales);
    static constexpr int kTiles = NQ == 1 ? 2 : 1;      // tiles of a warp at a time
    static constexpr int kStages = (D == 128 ? 3 : 7) + kTiles;
    static constexpr int kRows = 8 * NQ;
    static constexpr int kRing = kAttnWarps * kStages * kStage;
    // queries in the order of the products, then what rows and warps exchange
    static constexpr int kQBytes = D / 16 * NQ * 32 * 8;
    // a warp's scales: the keys' in fp32, the values' for pairs of tokens
    static constexpr int kScaleWords = (kAttnTile + kAttnTile / 2) * kBlocks;   // of a tile
    static constexpr int kScaleBytes = kTiles * kScaleWords * 4;
    static constexpr int kScaleAt = kRing + kQBytes;
    static constexpr int kSmem = kScaleAt + kAttnWarps * kScaleBytes + (kRows + 2 * kAttnWarps * kRows) * 4;
    static_assert(kAttnWarps * 8 * D * 4 <= kRing, "the warps' sums are exchanged where the ring was");
};

// 16-byte piece c of a tile's row r: where it lies in the row.
template <int D>
__host__ __device__ constexpr int swizzled(int r, int c) {
    return D == 128 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1);
}

// The first unit of each request (s_first[B]: all units), by the whole CTA.
__device__ __forceinline__ void plan_units(const AttnArgs &a, int rows_at_once, int *s_first, int *s_warp) {
    int before = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int units = 0;
        if (b < a.B) {
            const AttnRequest r = attn_request(a, b);
            const int tiles = (int)(((int64_t)r.n * a.G + rows_at_once - 1) / rows_at_once);
            const int64_t want = (int64_t)a.Hk * tiles * (attn_chunks(r) + kPieceUnits);
            // all requests together stay within 31 bits, and CTAs' shares of them within 32
            const bool few = (int64_t)r.n * a.G <= a.few_rows;   // else another kernel's
            units = few && want <= (1 << 30) / a.B ? (int)want : 0;
            if ((r.bad || (few && units != want)) && blockIdx.x == 0 && a.status) atomicOr(a.status, MOE_DEV_BAD_INDEX);
        }
        int v = units;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = v;
        __syncthreads();
        int sum = before;
        for (int w = 0; w < kAttnWarps; ++w) {
            if (w < warp) v += s_warp[w];
            sum += s_warp[w];
        }
        if (b < a.B) s_first[b] = before + v - units;
        before = sum;
    }
    if (threadIdx.x == 0) s_first[a.B] = before;
    __syncthreads();
}

// Four channels of the output, times inv.
__device__ __forceinline__ void write4(const AttnArgs &a, int64_t at, const float4 v, float inv) {
    if (a.out_bf16) {
        const __nv_bfloat162 y0 = __floats2bfloat162_rn(v.x * inv, v.y * inv);
        const __nv_bfloat162 y1 = __floats2bfloat162_rn(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&y0), *reinterpret_cast<const uint32_t *>(&y1));
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) =
            make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    }
}

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, NQ == 4 ? 1 : 2) attention4_kernel(const AttnArgs a) {
    using S = Shape<D, NQ>;
    constexpr int kBlocks = S::kBlocks, kTiles = S::kTiles;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_warp[kAttnWarps];
    uint2 *s_q = reinterpret_cast<uint2 *>(smem + S::kRing);                 // [k step][8 rows][lane]
    float *s_ks = reinterpret_cast<float *>(smem + S::kScaleAt + (threadIdx.x >> 5) * S::kScaleBytes);   // [token][block]
    uint32_t *s_vs = reinterpret_cast<uint32_t *>(s_ks) + kAttnTile * kBlocks;                           // [pair][block]
    float *s_mult = reinterpret_cast<float *>(smem + S::kScaleAt + kAttnWarps * S::kScaleBytes);   // [rows]
    float *s_top = s_mult + S::kRows, *s_sum = s_top + kAttnWarps * S::kRows;  // [warp][rows]
    int *s_first = reinterpret_cast<int *>(smem + S::kSmem);                 // [requests + 1]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    pdl_launch_dependents();
    pdl_wait();
    plan_units(a, S::kRows, s_first, s_warp);
    // (as many units as a warp's tiles at a time: fewer take as long)
    const int all = s_first[a.B], per = max(S::kTiles, (all + (int)gridDim.x - 1) / (int)gridDim.x);
    if (tid == 0) a.cuts[blockIdx.x].nrows = 0;
    int u = min(all, (int)blockIdx.x * per);
    const int u_end = min(all, u + per);
    uint8_t *ring = smem + warp * S::kStages * S::kStage;
    const uint32_t ring_addr = smem_u32(ring);

    // The pieces of the CTA's units, one after the other: request b, KV head h, row group
    // qt, units c0 .. c1-1 of `chunks`.  Found by a search once: the code of a search, and
    // its divisions, waited 2000 cycles for instructions at each piece.
    int b = 0, h = 0, qt = 0, x0 = 0, chunks = 0, tiles_q = 0;
    AttnRequest r = {};
    auto take = [&]() {
        r = attn_request(a, b);
        chunks = attn_chunks(r);
        tiles_q = (int)(((int64_t)r.n * a.G + S::kRows - 1) / S::kRows);
    };
    if (u < u_end) {
        int hi = a.B;
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (s_first[mid] <= u) b = mid;
            else hi = mid;
        }
        take();
        const int local = u - s_first[b], piece = local / (chunks + kPieceUnits);
        x0 = local - piece * (chunks + kPieceUnits);
        h = piece / tiles_q, qt = piece - h * tiles_q;
    }
    auto advance = [&]() {
        x0 = 0;
        if (++qt < tiles_q) return;
        qt = 0;
        if (++h < a.Hk) return;
        h = 0;
        do ++b;
        while (s_first[b + 1] <= u);
        take();
    };
    for (; u < u_end; u < u_end ? advance() : void()) {
        const int x1 = min(chunks + kPieceUnits, x0 + u_end - u), last_unit = u - x0 + chunks + kPieceUnits - 1;
        const int c0 = max(0, x0 - kPieceUnits), c1 = max(0, x1 - kPieceUnits);
        u += x1 - x0;
        if (c0 == c1) continue;
        // the query token of a row of the request
        auto token_of = [&](int row) { return r.n == 1 ? 0 : row / a.G; };
        const int pos0 = r.len - r.n;                     // position of the request's first row
        const int rowbase = qt * S::kRows;                // (query token, head) rows, token-major
        const int nrows = min(S::kRows, r.n * a.G - rowbase);
        const int pos_lo = pos0 + token_of(rowbase), pos_hi = pos0 + token_of(rowbase + nrows - 1);
        const int t_end = min(r.lo + c1 * kAttnChunk, pos_hi + 1);   // tokens seen by any of these rows
        const int t_begin = r.lo + c0 * kAttnChunk;

        // ---- this warp's tiles: t_begin + 16 (warp + 8 i)
        const int first_tile = t_begin + warp * kAttnTile;
        const int ntiles = first_tile < t_end ? (t_end - first_tile + kAttnChunk - 1) / kAttnChunk : 0;
        int ids = -1;         // lane i: the page of the warp's tile 32 k + i
        uint32_t there = 0;   // bit 0: the tile last fetched has a page, bit 1: the one before, ...
        uint32_t to = 0;      // the slot that the next tile goes to
        constexpr int kPieces = S::kCodes / 16, kInRow = S::kRow / 16;   // 16-byte pieces of a tile and of a row
        constexpr int kScalePieces = S::kScales / 16;
        // Where this lane's pieces come from (in page 0) and go to (in a slot).  The warp's
        // tiles are a multiple of a page apart, so they lie alike in their pages.
        static_assert(kAttnChunk % 128 == 0, "pages of 16 to 128 tokens");
        const int64_t kv_rows = (int64_t)a.Hk << a.page_shift;
        const int64_t row0 = ((int64_t)h << a.page_shift) + (first_tile & ((1 << a.page_shift) - 1));
        const uint32_t page_codes = (uint32_t)(2 * kv_rows * S::kRow), page_scales = (uint32_t)(2 * kv_rows * kBlocks);
        const uint8_t *src_k = a.codes + row0 * S::kRow + (lane % kPieces) * 16, *src_v = src_k + kv_rows * S::kRow;
        const uint8_t *src_s = a.scales + (row0 + (lane / kScalePieces) * kv_rows) * kBlocks + lane % kScalePieces * 16;
        const int piece_row = lane / kInRow;
        const uint32_t dst = ring_addr + piece_row * S::kRow + swizzled<D>(piece_row, lane % kInRow) * 16;
        static_assert(swizzled<D>(0, 1) == swizzled<D>(32 / kInRow, 1), "the pieces 32 apart lie alike");
        // Copies tile i into its slot of the ring; a page that is not there
        // leaves the slot as it is (its tokens are not seen).
        auto fetch = [&](int i) {
            there <<= 1;
            if (i < ntiles) {
                if ((i & 31) == 0) {
                    const int64_t t = first_tile + (int64_t)(i + lane) * kAttnChunk;
                    ids = -1;
                    if (t < t_end) {
                        ids = a.table[(int64_t)b * a.max_pages + (t >> a.page_shift)];
                        if (ids < 0 || ids >= a.pages) {
                            if (a.status) atomicOr(a.status, MOE_DEV_BAD_INDEX);
                            ids = -1;
                        }
                    }
                }
                const int id = __shfl_sync(0xffffffffu, ids, i & 31);
                if (id >= 0) {
                    there |= 1u;
                    const uint64_t page_at = (uint64_t)(uint32_t)id * page_codes;
                    const uint8_t *k = src_k + page_at, *v = src_v + page_at;
#pragma unroll
                    for (int j = 0; j < kPieces; j += 32) {
                        cp_async16(dst + to + j * 16, k + j * 16);
                        cp_async16(dst + to + S::kCodes + j * 16, v + j * 16);
                    }
                    if (lane < 2 * kScalePieces)
                        cp_async16(ring_addr + to + 2 * S::kCodes + lane * 16, src_s + (uint64_t)(uint32_t)id * page_scales);
                }
            }
            cp_async_commit();
            to = to == (S::kStages - 1) * S::kStage ? 0 : to + S::kStage;
        };
        // The queries of rows warp, warp + 8 .. on their way before page ids are waited for
        // (after them: 48 requests 64.9 us for 62.1).
        static_assert(kAttnWarps == 8, "a warp's rows are eight apart");
        uint2 raw[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int rr = warp + 8 * n, row = rowbase + rr;
            raw[n] = make_uint2(0, 0);
            if (rr < nrows) {
                const int token = token_of(row);
                const uint16_t *q = a.q + ((int64_t)(r.row0 + token) * a.Hq + h * a.G + row - token * a.G) * D;
                if (D == 128) raw[n] = reinterpret_cast<const uint2 *>(q)[lane];
                else raw[n].x = reinterpret_cast<const uint32_t *>(q)[lane];
            }
        }
#pragma unroll
        for (int i = 0; i < S::kStages - kTiles; ++i) fetch(i);

        // ---- queries: fp16 in the order of the products, a power of two for each row
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int rr = warp + 8 * n;
            float v[D / 32];
            float amax = 0.0f;
            v[0] = __uint_as_float(raw[n].x << 16), v[1] = __uint_as_float(raw[n].x & 0xffff0000u);
            if (D == 128)
                v[2 % (D / 32)] = __uint_as_float(raw[n].y << 16), v[3 % (D / 32)] = __uint_as_float(raw[n].y & 0xffff0000u);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) amax = fmaxf(amax, fabsf(v[j]));
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            // amax 2^up in [2^14, 2^15); the exponent is held where 2^up is a number
            const int ex = (int)(__float_as_uint(amax) >> 23);
            const int up = 14 + 127 - min(max(ex, 27), 254);
            const float f = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) v[j] *= f;
            if (lane == 0) s_mult[rr] = a.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
            // Channel 32 b + 8 c + 4 s + {0,1 | 2,3} of row (n, g) is word {0 | 1} of
            // lane (g, c) in step 2 b + s
            uint32_t *dst = reinterpret_cast<uint32_t *>(s_q);
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const int ch = lane * (D / 32) + 2 * j;
                const int blk = ch >> 5, cc = (ch >> 3) & 3, st = (ch >> 2) & 1, word = (ch >> 1) & 1;
                dst[(((2 * blk + st) * NQ + n) * 32 + warp * 4 + cc) * 2 + word] = half2_bits(v[2 * j], v[2 * j + 1]);
            }
        }
        __syncthreads();

        // ---- the pass over the tokens
        uint2 qf[NQ == 1 ? D / 16 : 1][NQ];
        if (NQ == 1)
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int n = 0; n < NQ; ++n) qf[k][n] = s_q[(k * NQ + n) * 32 + lane];
        float mult[NQ][2], ref[NQ][2], sum[NQ][2];   // ref: m - 11, 0 before there is one
        int last[NQ][2];   // position of this lane's two rows (columns of the products)
        float o[2 * kBlocks][NQ][4];
        float pass[NQ][2];         // what may pass ref: kAttnTop, or nothing before there is an m
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int rr = 8 * n + 2 * c + j;
                mult[n][j] = s_mult[rr];
                pass[n][j] = -INFINITY;
                ref[n][j] = 0.0f;
                sum[n][j] = 0.0f;
                last[n][j] = pos0 + token_of(rowbase + min(rr, nrows - 1));
            }
#pragma unroll
        for (int m = 0; m < 2 * kBlocks; ++m)
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[m][n][j] = 0.0f;
        // ldmatrix rows of this lane: row lane % 8 (+ 8 for the odd matrices) of pieces
        // (blocks) 2 x + lane / 16
        const int mrow = (lane & 7) + ((lane >> 3) & 1) * 8, mblk = lane >> 4;

        uint32_t from = 0;   // the slot of tile i
        for (int i = 0; i < ntiles; i += kTiles) {
            cp_async_wait<S::kStages - 2 * kTiles>();
            __syncwarp();
#pragma unroll
            for (int u = 0; u < kTiles; ++u) fetch(i + S::kStages - kTiles + u);   // into the slots of the tiles before
            uint32_t slot[kTiles];
#pragma unroll
            for (int u = 0; u < kTiles; ++u) {
                slot[u] = from;
                from = from == (S::kStages - 1) * S::kStage ? 0 : from + S::kStage;
            }
            // which of the tiles are there: all of them, but for the last round and bad pages
            const uint32_t have = there >> (S::kStages - kTiles);
            if ((have & ((1u << kTiles) - 1)) == 0) continue;
            const int t0 = first_tile + i * kAttnChunk;   // tile u: t0 + u kAttnChunk
            const bool edge = t0 + (kTiles - 1) * kAttnChunk + kAttnTile - 1 > pos_lo ||
                              (a.window && t0 <= pos_hi - a.window) || (~have & ((1u << kTiles) - 1));
            // Scales, each formed by one lane.  Keys: 2^(byte - 127) in fp32; byte 0 (2^-127) counts as
            // zero, 255 as infinity: its codes are zero, and zero times it NaN.
            const int vp = (lane / kBlocks) & 7, vk = lane % kBlocks;   // values: tokens 2 vp, 2 vp + 1 of block vk
            // (a tile's bytes for this lane's pair: what no row sees, written to or not, as any other)
            auto value_bytes = [&](int u, uint32_t &e0, uint32_t &e1) {
                const uint8_t *sv = ring + slot[u] + 2 * S::kCodes + S::kScales + 2 * vp * kBlocks + vk;
                e0 = sv[0], e1 = sv[kBlocks];
                if (edge) {
                    const int t = t0 + u * kAttnChunk + 2 * vp, seen = a.window ? pos_lo - a.window : -1;
                    const bool gone = !(have >> (kTiles - 1 - u) & 1u);
                    if (gone || t > pos_hi || t <= seen) e0 = 127u;
                    if (gone || t + 1 > pos_hi || t + 1 <= seen) e1 = 127u;
                }
            };
            bool odd = false;   // a value's scale beyond fp16's
#pragma unroll
            for (int u = 0; u < kTiles; ++u) {
                const uint8_t *sc = ring + slot[u] + 2 * S::kCodes;
                if (kBlocks == 4) {
                    const uint32_t w = reinterpret_cast<const uint16_t *>(sc)[lane];
                    reinterpret_cast<uint2 *>(s_ks + u * S::kScaleWords)[lane] = make_uint2((w & 0xffu) << 23, w >> 8 << 23);
                } else {
                    s_ks[u * S::kScaleWords + lane] = __uint_as_float((uint32_t)sc[lane] << 23);
                }
                uint32_t e0, e1;
                value_bytes(u, e0, e1);
                odd |= e0 - kLeastHalf >= kBand || e1 - kLeastHalf >= kBand;
                s_vs[u * S::kScaleWords + vp * kBlocks + vk] = half2_bits(__uint_as_float(e0 << 23), __uint_as_float(e1 << 23));
            }
            odd = __any_sync(0xffffffffu, odd);
            // Band k: scale bytes kLeastHalf + k kBand .., as 2^(e - 127 - k kBand); 0 what is not in it
            auto band_scale = [](uint32_t e, int k) {
                const uint32_t from = e - (uint32_t)(kLeastHalf + k * kBand);
                return e != 255u && from < kBand ? __uint_as_float((from + kLeastHalf) << 23) : 0.0f;
            };
            if (odd) {   // band 0 alone
#pragma unroll
                for (int u = 0; u < kTiles; ++u) {
                    uint32_t e0, e1;
                    value_bytes(u, e0, e1);
                    s_vs[u * S::kScaleWords + vp * kBlocks + vk] = half2_bits(band_scale(e0, 0), band_scale(e1, 0));
                }
            }
            __syncwarp();
            // S^T = K Q^T
            float s[kTiles][NQ][4];
#pragma unroll
            for (int u = 0; u < kTiles; ++u) {
                float ks0[kBlocks], ks1[kBlocks];   // of tokens g and g + 8
                load_blocks<kBlocks>(ks0, s_ks + u * S::kScaleWords + g * kBlocks);
                load_blocks<kBlocks>(ks1, s_ks + u * S::kScaleWords + (g + 8) * kBlocks);
#pragma unroll
                for (int x = 0; x < kBlocks / 2; ++x) {
                    uint32_t w[4];   // tokens 0-7 and 8-15 of block 2 x, then of block 2 x + 1
                    ldm4(ring_addr + slot[u] + mrow * S::kRow + swizzled<D>(mrow, 2 * x + mblk) * 16, w);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int k = 2 * x + y;
                        uint32_t k0[4], k1[4];
                        mx4_half8(w[2 * y], k0);
                        mx4_half8(w[2 * y + 1], k1);
                        const float f0 = ks0[k], f1 = ks1[k];
#pragma unroll
                        for (int n = 0; n < NQ; ++n) {
                            float d[4];
                            const uint2 qa = NQ == 1 ? qf[NQ == 1 ? 2 * k : 0][n] : s_q[(2 * k * NQ + n) * 32 + lane];
                            const uint2 qb = NQ == 1 ? qf[NQ == 1 ? 2 * k + 1 : 0][n]
                                                     : s_q[((2 * k + 1) * NQ + n) * 32 + lane];
                            mma16816_first(d, k0[0], k1[0], k0[1], k1[1], qa.x, qa.y);
                            mma16816(d, k0[2], k1[2], k0[3], k1[3], qb.x, qb.y);
                            s[u][n][0] = k ? fmaf(d[0], f0, s[u][n][0]) : d[0] * f0;
                            s[u][n][1] = k ? fmaf(d[1], f0, s[u][n][1]) : d[1] * f0;
                            s[u][n][2] = k ? fmaf(d[2], f1, s[u][n][2]) : d[2] * f1;
                            s[u][n][3] = k ? fmaf(d[3], f1, s[u][n][3]) : d[3] * f1;
                        }
                    }
                }
            }
            // scores past the maximum, masked; rows of s: tokens t0 + g and t0 + g + 8
            bool over = false;
#pragma unroll
            for (int u = 0; u < kTiles; ++u)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[u][n][j] = fmaf(s[u][n][j], mult[n][j & 1], -ref[n][j & 1]);
            if (edge) {
#pragma unroll
                for (int u = 0; u < kTiles; ++u)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int t = t0 + u * kAttnChunk + g + (j >> 1) * 8, p = last[n][j & 1];
                            if (t > p || (a.window && t <= p - a.window) || !(have >> (kTiles - 1 - u) & 1u))
                                s[u][n][j] = -INFINITY;
                        }
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v = fmaxf(s[0][n][j], s[0][n][j + 2]);
#pragma unroll
                    for (int u = 1; u < kTiles; ++u) v = fmaxf(v, fmaxf(s[u][n][j], s[u][n][j + 2]));
                    over |= v > pass[n][j];
                }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float v = fmaxf(s[0][n][j], s[0][n][j + 2]);
#pragma unroll
                        for (int u = 1; u < kTiles; ++u) v = fmaxf(v, fmaxf(s[u][n][j], s[u][n][j + 2]));
#pragma unroll
                        for (int x = 4; x <= 16; x <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
                        // how far m moves
                        const float up = v == -INFINITY ? 0.0f : pass[n][j] == -INFINITY ? v - kRest : fmaxf(v - kRest, 0.0f);
                        // before there is an m there is nothing to scale
                        const float f = pass[n][j] == -INFINITY ? 1.0f : ex2(-up);
                        if (v != -INFINITY) pass[n][j] = kAttnTop;
                        ref[n][j] += up;
                        sum[n][j] *= f;
#pragma unroll
                        for (int u = 0; u < kTiles; ++u) s[u][n][j] -= up, s[u][n][j + 2] -= up;
#pragma unroll
                        for (int m = 0; m < 2 * kBlocks; ++m) o[m][n][j] *= f, o[m][n][j + 2] *= f;
                    }
            }
#pragma unroll
            for (int u = 0; u < kTiles; ++u) {
                // P^T, transposed into the order of the second product
                uint32_t pt[NQ][2];
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    float p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[j] = ex2(s[u][n][j]);
                        sum[n][j & 1] += p[j];
                    }
                    pt[n][0] = transposed8(half2_bits(p[0], p[1]));
                    pt[n][1] = transposed8(half2_bits(p[2], p[3]));
                }
                // Values of a tile, channel block k: of channels 4g .. 4g+3 of token 2c in the low half
                // of the word, of token 2c + 1 in the high half (+ 8 in the second word)
                auto values = [&](const uint32_t (&w)[4], int y, uint32_t f0, uint32_t f1, uint32_t (&v0)[4], uint32_t (&v1)[4]) {
                    mx4_half8(token_pairs(w[2 * y]), v0);
                    mx4_half8(token_pairs(w[2 * y + 1]), v1);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v0[j] = mul_half2(v0[j], f0), v1[j] = mul_half2(v1[j], f1);
                };
                const uint32_t values_at = ring_addr + slot[u] + S::kCodes + mrow * S::kRow;
                // the values' scales of tokens 2c, 2c+1 and 2c+8, 2c+9
                uint32_t *const scales = s_vs + u * S::kScaleWords;
                uint32_t vs0[kBlocks], vs1[kBlocks];
                load_blocks<kBlocks>(vs0, scales + c * kBlocks);
                load_blocks<kBlocks>(vs1, scales + (c + 4) * kBlocks);
                // O^T += V^T P^T
#pragma unroll
                for (int x = 0; x < kBlocks / 2; ++x) {
                    uint32_t w[4];
                    ldm4_trans(values_at + swizzled<D>(mrow, 2 * x + mblk) * 16, w);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int k = 2 * x + y;
                        uint32_t v0[4], v1[4];
                        values(w, y, vs0[k], vs1[k], v0, v1);
#pragma unroll
                        for (int n = 0; n < NQ; ++n) {
                            mma16816(o[2 * k][n], v0[0], v0[2], v1[0], v1[2], pt[n][0], pt[n][1]);       // channels 4g, 4g + 1
                            mma16816(o[2 * k + 1][n], v0[1], v0[3], v1[1], v1[3], pt[n][0], pt[n][1]);   // 4g + 2, 4g + 3
                        }
                    }
                }
                if (!odd) continue;
                uint32_t e0, e1;
                value_bytes(u, e0, e1);
#pragma unroll 1
                for (int band = -3; band <= 4; ++band) {
                    const float s0 = band_scale(e0, band), s1 = band_scale(e1, band);
                    if (band == 0 || !__any_sync(0xffffffffu, s0 != 0.0f || s1 != 0.0f)) continue;
                    __syncwarp();   // the scales before have been read
                    scales[vp * kBlocks + vk] = half2_bits(s0, s1);
                    __syncwarp();
                    load_blocks<kBlocks>(vs0, scales + c * kBlocks);
                    load_blocks<kBlocks>(vs1, scales + (c + 4) * kBlocks);
                    // 2^(band kBand), which fp32 does not have for all bands: as two
                    const float fa = __uint_as_float((uint32_t)(127 + band * (kBand / 2)) << 23);
                    const float fb = __uint_as_float((uint32_t)(127 + band * (kBand - kBand / 2)) << 23);
#pragma unroll
                    for (int x = 0; x < kBlocks / 2; ++x) {
                        uint32_t w[4];
                        ldm4_trans(values_at + swizzled<D>(mrow, 2 * x + mblk) * 16, w);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int k = 2 * x + y;
                            uint32_t v0[4], v1[4];
                            values(w, y, vs0[k], vs1[k], v0, v1);
#pragma unroll
                            for (int n = 0; n < NQ; ++n) {
                                float d0[4], d1[4];
                                mma16816_first(d0, v0[0], v0[2], v1[0], v1[2], pt[n][0], pt[n][1]);
                                mma16816_first(d1, v0[1], v0[3], v1[1], v1[3], pt[n][0], pt[n][1]);
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    o[2 * k][n][j] += d0[j] * fa * fb, o[2 * k + 1][n][j] += d1[j] * fa * fb;
                            }
                        }
                    }
                }
                // what is NaN: the scales' place has a mark for it now
                const uint32_t marks = (e0 == 255u ? kNan : 0u) | (e1 == 255u ? kNan << 16 : 0u);
                const bool nans = __any_sync(0xffffffffu, marks != 0);
                __syncwarp();
                scales[vp * kBlocks + vk] = marks;
                __syncwarp();
                load_blocks<kBlocks>(vs0, scales + c * kBlocks);
                load_blocks<kBlocks>(vs1, scales + (c + 4) * kBlocks);
                if (nans) {   // NaN for the rows that see it (not by P, which fp16 may have made zero), in its block
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        uint32_t seen[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            seen[j] = transposed8((s[u][n][2 * j] == -INFINITY ? 0u : 1u) | (s[u][n][2 * j + 1] == -INFINITY ? 0u : 1u << 16));
#pragma unroll
                        for (int k = 0; k < kBlocks; ++k) {
                            const bool hit = sees_nan(seen[0], vs0[k]) || sees_nan(seen[1], vs1[k]);
                            const uint32_t lanes = __ballot_sync(0xffffffffu, hit);   // four lanes to row g
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (lanes >> (8 * c + 4 * j) & 15u)
                                    o[2 * k][n][j] = o[2 * k][n][j + 2] = o[2 * k + 1][n][j] = o[2 * k + 1][n][j + 2] = NAN;
                        }
                    }
                }
            }
        }

        // ---- the warps' results together
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) sum[n][j] += __shfl_xor_sync(0xffffffffu, sum[n][j], x);
                if (g == 0) {
                    s_top[warp * S::kRows + 8 * n + 2 * c + j] = pass[n][j] == -INFINITY ? -INFINITY : ref[n][j];
                    s_sum[warp * S::kRows + 8 * n + 2 * c + j] = sum[n][j];
                }
            }
        cp_async_wait<0>();
        __syncthreads();   // the ring is free, and the maxima are there
        const bool whole = c0 == 0 && c1 == chunks;
        if (tid == 0 && c0 == 0 && !whole) {
            const AttnCut cut = {r.row0, h * a.G, rowbase, nrows, last_unit / per, {}};
            a.cuts[blockIdx.x] = cut;
        }
        float *part = a.part + (int64_t)(2 * blockIdx.x + (c0 == 0 ? 1 : 0)) * S::kRows * (D + 2);
        float *s_o = reinterpret_cast<float *>(smem);   // [warp][8 rows][D]
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int rr = 8 * n + 2 * c + j;
                float m = s_top[rr];
#pragma unroll
                for (int w = 1; w < kAttnWarps; ++w) m = fmaxf(m, s_top[w * S::kRows + rr]);
                const float mine = s_top[warp * S::kRows + rr], f = mine == m ? 1.0f : ex2(mine - m);
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) {
                    *reinterpret_cast<float4 *>(s_o + ((warp * 8 + 2 * c + j) * D + 32 * k + 4 * g)) =
                        make_float4(o[2 * k][n][j] * f, o[2 * k][n][j + 2] * f, o[2 * k + 1][n][j] * f,
                                    o[2 * k + 1][n][j + 2] * f);
                }
            }
            __syncthreads();
            for (int x = tid; x < 8 * D / 4; x += kThreads) {
                const int rr = 8 * n + x / (D / 4), col = x % (D / 4) * 4;
                float m = s_top[rr], l = 0.0f;
#pragma unroll
                for (int w = 1; w < kAttnWarps; ++w) m = fmaxf(m, s_top[w * S::kRows + rr]);
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kAttnWarps; ++w) {
                    const float tw = s_top[w * S::kRows + rr];
                    l += s_sum[w * S::kRows + rr] * (tw == m ? 1.0f : ex2(tw - m));
                    const float4 y = *reinterpret_cast<const float4 *>(s_o + (w * 8 + x / (D / 4)) * D + col);
                    v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
                }
                if (!whole) {
                    *reinterpret_cast<float4 *>(part + rr * D + col) = v;
                    if (col == 0) part[S::kRows * D + rr] = m, part[S::kRows * (D + 1) + rr] = l;
                } else if (rr < nrows) {
                    const int row = rowbase + rr, token = token_of(row);
                    const int64_t at = (int64_t)(r.row0 + token) * a.Hq + h * a.G + row - token * a.G;
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // a row that sees nothing
                    write4(a, at * D + col, v, inv);
                    if (a.lse && col == 0) a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
                }
            }
            __syncthreads();
        }
    }
}

// One block: eight rows of what CTA blockIdx.x began.  A warp takes one of them, eight
// partial results on their way at a time; where there are more than 32, every eighth for
// all of the rows.  (All ways like that: one request 13.9 us for 11.4, two long ones 101.8
// for 98, 48 requests, mostly of two partial results, 64.3 for 64.9.)
constexpr int kJoinRows = 8, kShortJoin = 32, kJoinAhead = 8;

template <int D>
__global__ void __launch_bounds__(256, 3) attention4_join_kernel(const AttnArgs a, int rows_at_once) {
    constexpr int V = D / 32;   // channels of a lane
    __shared__ float s_top[8][kJoinRows], s_sum[8][kJoinRows];
    __shared__ __align__(16) float s_o[8][kJoinRows][D];
    pdl_launch_dependents();
    pdl_wait();
    const int k0 = blockIdx.x, r0 = blockIdx.y * kJoinRows, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const AttnCut cut = a.cuts[k0];
    if (r0 >= cut.nrows) return;
    const int parts = cut.last - k0 + 1;
    const int64_t size = (int64_t)rows_at_once * (D + 2);
    auto part = [&](int j) { return a.part + (2 * (int64_t)(k0 + j) + (j == 0)) * size; };
    if (parts <= kShortJoin) {   // a warp to a row, a lane to each partial's maximum and sum
        const int rr = r0 + warp;
        if (rr >= cut.nrows) return;
        const bool mine = lane < parts, writes = lane < D / 4;
        float4 y[kJoinAhead];
        auto load = [&](int j0) {
#pragma unroll
            for (int j = 0; j < kJoinAhead; ++j)
                if (j0 + j < parts && writes) y[j] = *reinterpret_cast<const float4 *>(part(j0 + j) + (int64_t)rr * D + 4 * lane);
        };
        load(0);
        const float *p = part(mine ? lane : 0) + rows_at_once * D + rr;
        const float m = mine ? p[0] : -INFINITY;
        float l = mine ? p[rows_at_once] : 0.0f, top = m;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float f = m == top ? 1.0f : ex2(m - top);
        l *= f;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
        for (int j0 = 0; j0 < parts; j0 += kJoinAhead) {
#pragma unroll
            for (int j = 0; j < kJoinAhead; ++j) {
                const float fj = __shfl_sync(0xffffffffu, f, (j0 + j) & 31);
                if (j0 + j < parts && writes) v.x += fj * y[j].x, v.y += fj * y[j].y, v.z += fj * y[j].z, v.w += fj * y[j].w;
            }
            load(j0 + kJoinAhead);
        }
        const int row = cut.rowbase + rr;
        const int64_t at = (int64_t)(cut.row0 + row / a.G) * a.Hq + cut.head0 + row % a.G;
        if (writes) write4(a, at * D + 4 * lane, v, l == 0.0f ? 0.0f : 1.0f / l);
        if (a.lse && lane == 0) a.lse[at] = l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.69314718f;
        return;
    }
    {   // each row's largest: lane rr + 8 i of a warp takes partial 4 warp + i + 32 n
        float m = -INFINITY;
        for (int j = 4 * warp + (lane >> 3); j < parts; j += 32)
            m = fmaxf(m, part(j)[rows_at_once * D + r0 + (lane & 7)]);
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (lane < kJoinRows) s_top[warp][lane] = m;
    }
    __syncthreads();
    float top = s_top[0][lane & 7];   // of row lane % 8
#pragma unroll
    for (int w = 1; w < 8; ++w) top = fmaxf(top, s_top[w][lane & 7]);
    float o[kJoinRows][V], sum = 0.0f;
#pragma unroll
    for (int rr = 0; rr < kJoinRows; ++rr)
#pragma unroll
        for (int j = 0; j < V; ++j) o[rr][j] = 0.0f;
#pragma unroll 2
    for (int j = warp; j < parts; j += 8) {
        const float *p = part(j);
        const float m = p[rows_at_once * D + r0 + (lane & 7)];
        const float f = m == top ? 1.0f : ex2(m - top);
        sum += f * p[rows_at_once * (D + 1) + r0 + (lane & 7)];
#pragma unroll
        for (int rr = 0; rr < kJoinRows; ++rr) {
            const float fr = __shfl_sync(0xffffffffu, f, rr);
            if (r0 + rr >= cut.nrows) continue;
            const float *y = p + (int64_t)(r0 + rr) * D + lane * V;
            if (V == 4) {
                const float4 q = *reinterpret_cast<const float4 *>(y);
                o[rr][0] += fr * q.x, o[rr][1] += fr * q.y, o[rr][2 % V] += fr * q.z, o[rr][3 % V] += fr * q.w;
            } else {
                const float2 q = *reinterpret_cast<const float2 *>(y);
                o[rr][0] += fr * q.x, o[rr][1] += fr * q.y;
            }
        }
    }
    if (lane < kJoinRows) s_sum[warp][lane] = sum;
#pragma unroll
    for (int rr = 0; rr < kJoinRows; ++rr)
#pragma unroll
        for (int j = 0; j < V; ++j) s_o[warp][rr][lane * V + j] = o[rr][j];
    __syncthreads();
    for (int x = tid; x < kJoinRows * D / 4; x += 256) {
        const int rr = x / (D / 4), col = x % (D / 4) * 4;
        if (r0 + rr >= cut.nrows) break;
        float l = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            l += s_sum[w][rr];
            const float4 y = *reinterpret_cast<const float4 *>(&s_o[w][rr][col]);
            v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
        }
        const int row = cut.rowbase + r0 + rr;
        const int64_t at = (int64_t)(cut.row0 + row / a.G) * a.Hq + cut.head0 + row % a.G;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        write4(a, at * D + col, v, inv);
        if (a.lse && col == 0) {
            float m = s_top[0][rr];
#pragma unroll
            for (int w = 1; w < 8; ++w) m = fmaxf(m, s_top[w][rr]);
            a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
        }
    }
}

// Requests of at most this many rows are this file's where the call also has larger
// ones: up to there rows share a read of the cache here, and the other kernel's tiles
// would be a quarter full.  (16 requests of 4096 tokens, 64 query heads on 8, cold, in a
// graph: 32 rows 65 us here; 40 rows 107 here, 97 there; 128 rows 196 and 104.)
constexpr int kFewRows = 32;

int64_t most_rows(const moe_cache_attn *d, const moe_cache4 *cache) {
    return (int64_t)std::max(1, std::min(d->max_q, d->rows)) * (d->q_heads / cache->kv_heads);
}

bool has_wide(const moe_cache_attn *d, const moe_cache4 *cache) { return most_rows(d, cache) > kFewRows; }

// Groups of eight rows that a warp takes at once: as many as the largest request
// needs for its rows, four at most; where larger ones go elsewhere, as many as a
// query token needs.
int rows8(const moe_cache_attn *d, const moe_cache4 *cache) {
    const int64_t rows = has_wide(d, cache) ? d->q_heads / cache->kv_heads : most_rows(d, cache);
    return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}

template <int D, int NQ>
int launch(const AttnArgs &a0, cudaStream_t s) {
    using S = Shape<D, NQ>;
    AttnArgs a = a0;
    const int smem = S::kSmem + (a.B + 1) * 4;
    // (the most that any call takes: calls of several threads set the same)
    MOE_CUDA_TRY(cudaFuncSetAttribute(attention4_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      S::kSmem + (kAttnMaxRequests + 1) * 4));
    if (int rc = launch_dependent(attention4_kernel<D, NQ>, dim3(a.ctas), dim3(kThreads), smem, s, (const AttnArgs)a))
        return rc;
    return launch_attention4_join(a, D, S::kRows, a.ctas, s);
}

int ctas_of(int nq) { return sm_count() * (nq == 4 ? 1 : 2); }

// (of the most CTAs: a call of fewer rows takes no more than one of more)
size_t cuts_bytes() { return align_up(sizeof(AttnCut) * ctas_of(1)); }

}  // namespace

static size_t attention4_few_workspace(const moe_cache_attn *d, const moe_cache4 *cache) {
    const int nq = rows8(d, cache);
    return cuts_bytes() + align_up(sizeof(float) * 2 * (size_t)ctas_of(nq) * 8 * nq * (cache->dim + 2));
}

int launch_attention4_join(const AttnArgs &a, int dim, int rows_at_once, int ctas, cudaStream_t s) {
    const dim3 grid((unsigned)ctas, (unsigned)(rows_at_once / kJoinRows));
    if (dim == 64) return launch_dependent(attention4_join_kernel<64>, grid, dim3(256), 0, s, (const AttnArgs)a, rows_at_once);
    return launch_dependent(attention4_join_kernel<128>, grid, dim3(256), 0, s, (const AttnArgs)a, rows_at_once);
}

size_t attention4_workspace(const moe_cache_attn *d, const moe_cache4 *cache) {
    return attention4_few_workspace(d, cache) + (has_wide(d, cache) ? attention4_wide_workspace(d, cache) : 0);
}

int launch_attention4(const moe_cache_attn *d, const moe_cache4 *cache, const void *q, const int32_t *table,
                      const int32_t *lengths, const int32_t *starts, void *out, int out_dtype, float *lse,
                      void *ws, int32_t *status, cudaStream_t s) {
    AttnArgs a;
    a.q = static_cast<const uint16_t *>(q);
    a.codes = static_cast<const uint8_t *>(cache->codes);
    a.scales = static_cast<const uint8_t *>(cache->scales);
    a.table = table;
    a.lengths = lengths;
    a.starts = starts;
    a.out = out;
    a.lse = lse;
    a.status = status;
    a.B = d->requests;
    a.rows = d->rows;
    a.Hq = d->q_heads;
    a.Hk = cache->kv_heads;
    a.G = a.Hq / a.Hk;
    a.max_pages = d->max_pages;
    a.pages = cache->pages;
    a.page_shift = 0;
    while ((1 << a.page_shift) < cache->page) ++a.page_shift;
    // (a window of all that a request can hold is none)
    a.window = d->window >= (int64_t)d->max_pages * cache->page ? 0 : d->window;
    a.out_bf16 = out_dtype == MOE_OUT_BF16;
    a.scale_log2 = d->scale * 1.44269504f;
    const int nq = rows8(d, cache);
    const bool wide = has_wide(d, cache);
    // A single request that may have many rows is the other kernel's whatever it has: two launches
    // less (64 rows of 16 heads over 1024 tokens 22.7 us for 25.5).
    const bool few = !wide || a.B > 1;
    a.few_rows = !wide ? INT32_MAX : few ? kFewRows : 0;
    a.ctas = ctas_of(nq);
    a.cuts = static_cast<AttnCut *>(ws);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + cuts_bytes());
    if (few)
        if (int rc = cache->dim == 64 ? nq == 1 ? launch<64, 1>(a, s) : nq == 2 ? launch<64, 2>(a, s) : launch<64, 4>(a, s)
                     : nq == 1 ? launch<128, 1>(a, s) : nq == 2 ? launch<128, 2>(a, s) : launch<128, 4>(a, s))
            return rc;
    if (!wide) return MOE_OK;
    return launch_attention4_wide(a, d, cache, a.few_rows,
                                  static_cast<uint8_t *>(ws) + attention4_few_workspace(d, cache), s);
}

}  // namespace moe
