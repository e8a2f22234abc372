// Attention of many query rows over the four-bit cache (chunks of prompts), on
// the tensor cores' fifth-generation kinds:
//   S = Q K^T,  P = 2^(S - m + 7),  O += P V,  o = O / sum P
//
// A CTA takes 256 rows (query heads of one KV head, query tokens one after the
// other) as two tiles of 128, and passes over the keys and values in tiles of
// 128 tokens.  tcgen05.mma (fp32 in tensor memory): S from Q and K in shared
// memory, both bf16; O from P, fp16, which a tile's softmax leaves in tensor memory
// where S was, and V in shared memory with channels contiguous.  While one
// tile's softmax works on its S the products of the other are under way:
//   QK0 QK1 | PV0 QK0 PV1 QK1 | PV0 QK0 PV1 QK1 ...
// Warps 0-3 and 4-7 are the softmax of tile 0 and 1, a thread to a row; warps
// 8-11 unpack keys and values; warp 12 issues the products.
//
// A key's value, a code of two significant bits times a power of two, is a bf16 number
// whatever its scale, and so is q: S has no error but its sum's.  A value is an fp16 number where
// its scale is 2^-23 to 2^13.  A tile that has others takes its values as bf16, and P as two bf16
// numbers (16 bits) whose products follow one another: nothing depends on what a row does not see.
// m is raised only where a score passes it by 8 (in log2), so
// S is read once and O hardly ever; it rises by whole powers of two.  A value that is
// NaN counts as zero in the products; rows that see it remember its block.
//
// Work: one unit for each tile of tokens that a group of 256 rows sees (causal:
// fewer for earlier rows) and some for its beginning and end; each CTA takes as
// many neighbouring units as any other.  Rows cut between CTAs leave partial
// results, at most two groups a CTA, which a last kernel joins.
//
// Three prompts' chunks of 500 to 4096 tokens onto caches of up to 8192, 64 query
// heads on 8 of 128: 1242 us, 0.97 PFLOP/s, 51% of what a large library product
// reaches.  (1170 with keys and values relative to the largest of a tile and a piece: keys as bf16 cost 30 us, the
// second way for values and what P keeps where m rises 40, most of that by where code and registers
// then lie.)  What bounds it is the way from one half's S to its P (four rounds of load,
// exponentials, conversion, store: some 2500 cycles, then 1400 of waiting for the next S)
// against 1024 cycles of the other half's products: tensor
// memory is full (two S of 128 columns, two O), so there is no third tile to work on
// meanwhile.  (P in shared memory would free S sooner, but with both operands there
// products of 128 columns read 128 bytes a clock, all that it has.)
//
// Tiles of 64 tokens with two S each were slower (products of 64 columns take as long
// as of 128: 1.50 ms for 1.36), and so were 16 softmax warps with half a row to a thread
// (1.71: maxima and sums by shared memory); softmax in one piece of 128 columns
// spilled and left the instruction cache (3.0 ms; loops of 32 columns 1.85); largest
// scores looked for only where the sum of 32 probabilities is large (1.28 for 1.195:
// the sum is known last).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>

#include "attention4.cuh"
#include "mx4.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kWideRows = 256, kM = 128, kTok = 128;
constexpr int kSoftWarps = 8, kUnpackWarps = 4, kMmaWarp = kSoftWarps + kUnpackWarps;
constexpr int kWideThreads = (kMmaWarp + 1) * 32;
constexpr int kStages = 2, kInfos = 4;
constexpr int kTmemCols = 512;
// What the beginning and end of a piece cost, in tiles (with 2, 3, 4 and 6: 1330, 1250,
// 1194 and 1199 us where 4 and 6 tied).
constexpr int kPieceTiles = 5;
// Where a raised maximum is put (log2).  Raising it scales O and is dear: chunks of 4096, 500 and 2000 onto 8192, 4096
// and 6000 take 1179 us with scores of deviation 1, 1200 of 2 and 1374 of 4; with 11 instead 1208, 1388 and 1572.
constexpr float kRest = 7.0f;
constexpr uint32_t kLeastHalf = 104, kMostHalf = 140;   // scale bytes with which every code is an fp16 number

struct WideArgs {
    AttnArgs a;
    int few_rows, max_entries;
    int64_t *units;        // [entries + 1]: units before each (request, group of rows), of one head
    int64_t *per;          // units a CTA
    int32_t *entry_request, *first_entry;   // [entries], [requests + 1]
};

__device__ __forceinline__ uint32_t bf162_of(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ uint32_t mul_bf162(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Pairs of e2m1 values from fp16 to bf16, times 2^-112: all bits move down by three (such a value has none
// of the lowest three) and the sign goes back up, 2^12 + 7 2^12 = 2^15.
__device__ __forceinline__ uint32_t bf16_of_half2(uint32_t h) {
    const uint32_t t = h >> 3;
    return t + 7u * (t & 0x10001000u);
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Eight columns, there when it returns.
__device__ __forceinline__ void tmem_get8(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(addr)
        : "memory");
}
using F2 = uint64_t;   // two fp32 numbers
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// fp16 or bf16 operands, A K-major, B with channels contiguous
__host__ __device__ constexpr uint32_t idesc_mn(int M, int N, bool bf16) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (1u << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
// V: rows of 128 bytes (64 channels of a token), 128-byte swizzle; eight tokens 1024 bytes,
// the next 64 channels kTok rows on
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kTok * 128 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// A group of rows of a request: what it sees, in tiles.
struct RowGroup {
    int rowbase, nrows, pos_lo, pos_hi, lo, tiles;
};
__device__ __forceinline__ RowGroup row_group(const AttnArgs &a, const AttnRequest &r, int qt) {
    RowGroup w;
    w.rowbase = qt * kWideRows;
    w.nrows = (int)min((int64_t)kWideRows, (int64_t)r.n * a.G - w.rowbase);
    w.pos_lo = r.len - r.n + w.rowbase / a.G;
    w.pos_hi = r.len - r.n + (w.rowbase + w.nrows - 1) / a.G;
    w.lo = a.window && w.pos_lo >= a.window ? (w.pos_lo - a.window + 1) / kAttnTile * kAttnTile : 0;
    w.tiles = max(1, (w.pos_hi - w.lo + kTok) / kTok);   // pos_hi + 1 tokens
    return w;
}

// ---- the work list: one CTA -------------------------------------------------------------
__device__ __forceinline__ int64_t scan_add(int64_t v, int64_t *sh) {   // inclusive, over 1024 threads
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    int64_t x = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    const int64_t before = __shfl_sync(0xffffffffu, x, max(warp - 1, 0));
    return v + (warp > 0 ? before : 0);
}

__global__ void __launch_bounds__(1024) wide_plan_kernel(const WideArgs w, int ctas) {
    __shared__ int s_first[kAttnMaxRequests + 1];
    __shared__ int64_t sh[32], s_total;
    const AttnArgs &a = w.a;
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    int64_t before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 1024) {
        const int b = b0 + tid;
        int64_t groups = 0;
        if (b < a.B) {
            const AttnRequest r = attn_request(a, b);
            const int64_t rows = (int64_t)r.n * a.G;
            if (r.bad && a.status) atomicOr(a.status, MOE_DEV_BAD_INDEX);
            if (rows > w.few_rows) groups = (rows + kWideRows - 1) / kWideRows;
        }
        const int64_t v = scan_add(groups, sh);
        if (b < a.B) {
            // rows that more than one request claims: there is room for as many as there are rows
            s_first[b] = (int)min(before + v - groups, (int64_t)w.max_entries);
            w.first_entry[b] = s_first[b];
        }
        if (tid == 1023) s_total = v;
        __syncthreads();
        before += s_total;
        __syncthreads();
    }
    if (before > w.max_entries && tid == 0 && a.status) atomicOr(a.status, MOE_DEV_BAD_INDEX);
    const int entries = (int)min(before, (int64_t)w.max_entries);
    if (tid == 0) s_first[a.B] = w.first_entry[a.B] = entries;
    __syncthreads();
    int64_t units = 0;
    for (int e0 = 0; e0 < entries; e0 += 1024) {
        const int e = e0 + tid;
        int64_t n = 0;
        if (e < entries) {
            int lo = 0, hi = a.B;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_first[mid] <= e) lo = mid;
                else hi = mid;
            }
            w.entry_request[e] = lo;
            n = row_group(a, attn_request(a, lo), e - s_first[lo]).tiles + kPieceTiles;
        }
        const int64_t v = scan_add(n, sh);
        if (e < entries) w.units[e] = units + v - n;
        if (tid == 1023) s_total = v;
        __syncthreads();
        units += s_total;
        __syncthreads();
    }
    if (tid == 0) {
        w.units[entries] = units;
        w.per[0] = max((int64_t)1, (units * a.Hk + ctas - 1) / ctas);
    }
}

// ---- pieces -----------------------------------------------------------------------------
struct Piece {
    AttnRequest r;
    RowGroup g;
    int b, h, c0, c1;
};

// The pieces of units u .. u_end, one after the other: entry after entry, then
// the next head's.  Found by a search once.
struct Walk {
    int64_t u, u_end;
    int h, entry, at;   // at: units of the entry that are taken
    __device__ __forceinline__ void start(const WideArgs &w, int64_t first, int64_t end, int entries, int64_t total) {
        u = first, u_end = end;
        if (u >= u_end) return;
        h = (int)(u / total);
        const int64_t local = u - h * total;
        int lo = 0, hi = entries;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (w.units[mid] <= local) lo = mid;
            else hi = mid;
        }
        entry = lo;
        at = (int)(local - w.units[lo]);
    }
    // False when there are no more.  c0 == c1: nothing of the piece is computed here.
    __device__ __forceinline__ bool next(const WideArgs &w, int entries, Piece &p) {
        if (u >= u_end) return false;
        p.h = h;
        p.b = w.entry_request[entry];
        p.r = attn_request(w.a, p.b);
        p.g = row_group(w.a, p.r, entry - w.first_entry[p.b]);
        const int all = p.g.tiles + kPieceTiles, to = (int)min((int64_t)all, at + u_end - u);
        p.c0 = max(0, at - kPieceTiles);
        p.c1 = max(0, to - kPieceTiles);
        u += to - at;
        at = 0;
        if (++entry == entries) entry = 0, ++h;
        return true;
    }
};

struct Info {          // of a tile of tokens, from those who unpack it
    uint32_t bad;      // bit i: tokens 16 i .. are on a page that is not there
    uint32_t bf16;     // values are bf16, P is two numbers
    uint32_t nan;      // a value of the tile is NaN
};

template <int D>
struct WideShape {
    static constexpr int kHalf = kTok * 128;               // 128 rows of 64 channels
    static constexpr int kTileBytes = D / 64 * kHalf;      // Q of a tile, K or V of a stage
    static constexpr int kQ = 0, kK = 2 * kTileBytes, kV = kK + kStages * kTileBytes;
    static constexpr int kUsed = kV + kStages * kTileBytes + 1024;
    // one CTA on an SM: each takes all of the tensor memory
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    static constexpr int kO = 2 * kTok;                    // columns: S of both halves, then O
};

// A row's maximum, what may pass it, its sum, and what O is to be multiplied by.
struct RowState {
    float ref, pass, sum, shrink;
};

// P of a tile (scores at ts, this row's columns from < t <= upto, but for bad pages) as two bf16 numbers
// each: 16 columns become eight of the larger parts and eight of what they leave.  The largest score is
// looked for first, so that nothing has to be scaled.  A function of its own: in line it slowed the
// tiles that need none of it (prompts 1306 us for 1223; without any second way 1200).
__device__ __noinline__ RowState two_bf16(uint32_t ts, int upto, int from, uint32_t bad, float scale_log2, RowState r) {
    auto sixteen = [&](int k, float (&x)[16]) {
        uint32_t y[16];
        tmem_ld16(ts + 16 * k, y);
        tmem_wait_ld(y);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int t = 16 * k + i;
            x[i] = t <= upto && t > from && !(bad >> k & 1u) ? fmaf(__uint_as_float(y[i]), scale_log2, -r.ref) : -INFINITY;
        }
    };
    float top = -INFINITY, x[16];
#pragma unroll 1
    for (int k = 0; k < kTok / 16; ++k) {
        sixteen(k, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, x[i]);
    }
    if (top > r.pass) {
        const bool none = r.pass == -INFINITY;
        const float rise = none ? ceilf(top) - kRest : fmaxf(ceilf(top) - kRest, 0.0f), f = none ? 1.0f : ex2(-rise);
        r.pass = kAttnTop;
        r.ref += rise;
        r.sum *= f;
        r.shrink *= f;
    }
    F2 part = 0ull;
#pragma unroll 1
    for (int k = 0; k < kTok / 16; ++k) {
        uint32_t y[16];
        sixteen(k, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p0 = ex2(x[2 * i]), p1 = ex2(x[2 * i + 1]);
            part = add2(part, pack2(__float_as_uint(p0), __float_as_uint(p1)));
            y[i] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
            y[8 + i] = bf162_of(p0 - __uint_as_float(__float_as_uint(p0) & 0xffff0000u),
                                p1 - __uint_as_float(__float_as_uint(p1) & 0xffff0000u));
        }
        tmem_st16(ts + 16 * k, y);
    }
    r.sum += __uint_as_float((uint32_t)part) + __uint_as_float((uint32_t)(part >> 32));
    return r;
}

template <int D>
__global__ void __launch_bounds__(kWideThreads, 1) attention4_wide_kernel(const WideArgs w) {
    using S = WideShape<D>;
    constexpr int kBlocks = D / 32;
    extern __shared__ uint8_t dsmem[];
    __shared__ uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], info_full[kInfos];
    __shared__ uint64_t s_full[2], p_ready[2], q_full, o_full, drain_bar;
    __shared__ uint64_t e_full[2];
    __shared__ Info s_info[kInfos];
    __shared__ uint2 s_nan[kInfos][kTok / 2];        // a byte for each token and channel block
    __shared__ uint4 s_e[2][kUnpackWarps];           // each warp's bad pages, NaN, scales beyond fp16's
    __shared__ uint32_t tmem_slot;
    __shared__ int s_abort;
    const AttnArgs &a = w.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort_flag = &s_abort;
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&k_full[s]), kUnpackWarps);
            mbar_init(smem_u32(&v_full[s]), kUnpackWarps);
            mbar_init(smem_u32(&k_empty[s]), 1);
            mbar_init(smem_u32(&v_empty[s]), 1);
        }
        for (int s = 0; s < kInfos; ++s) mbar_init(smem_u32(&info_full[s]), kUnpackWarps);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&e_full[s]), kUnpackWarps);
            mbar_init(smem_u32(&s_full[s]), 1);
            mbar_init(smem_u32(&p_ready[s]), 4);
        }
        mbar_init(smem_u32(&q_full), kSoftWarps);
        mbar_init(smem_u32(&o_full), 1);
        mbar_init(smem_u32(&drain_bar), 1);
        s_abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t base = (smem_u32(dsmem) + 1023u) & ~1023u;
    uint8_t *smem = dsmem + (base - smem_u32(dsmem));
    const int entries = w.first_entry[a.B];
    const int64_t total = w.units[entries], all = total * a.Hk, per = w.per[0];
    if (tid == 0) a.cuts[blockIdx.x].nrows = 0;
    Walk walk;
    walk.start(w, min(all, (int64_t)blockIdx.x * per), min(all, (int64_t)(blockIdx.x + 1) * per), entries, total);
    Piece p;
    uint32_t tiles = 0, pieces = 0;   // counted by every role alike
    bool ok = true;
    // a wait of a whole warp
    auto wait = [&](uint64_t &bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_bounded(smem_u32(&bar), parity, abort_flag, a.status, MOE_DEV_TIMEOUT));
    };

    if (warp < kSoftWarps) {
        // ---- softmax, a thread to a row ---------------------------------------------------
        const int mt = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + mt * kTok, to = tmem + lanes + S::kO + mt * D;
        // 16-byte piece p of row r of the warp's 32 in shared memory, queries and then results; kLanes
        // lanes take a row together
        constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes;
        const int sub = lane / kLanes, piece = lane % kLanes;
        uint8_t *const rows32 = smem + S::kQ + mt * S::kTileBytes + (warp & 3) * 32 * 128;
        auto tile_piece = [&](int r, int p) { return rows32 + r * 128 + (p >> 3) * S::kHalf + (((p & 7) ^ (r & 7)) << 4); };
        uint32_t mine = 0;   // products' tiles of this half, of all pieces
        while (ok && walk.next(w, entries, p)) {
            if (p.c0 == p.c1) continue;
            const int rr = mt * kM + row, flat = p.g.rowbase + rr;
            const bool there = rr < p.g.nrows;
            const int64_t at = (int64_t)(p.r.row0 + flat / a.G) * a.Hq + p.h * a.G + flat % a.G;
            const int at_row = there ? (int)at : -1;   // (rows times heads stay within 32 bits)
            // The warp's 32 queries by kLanes lanes to a row: loads of whole rows, four on their way.
            // (A thread to a row took 12000 cycles a piece, 16 bytes of each line at a time; 4000 so.)
            uint4 next[4];
            auto load = [&](int i0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int src = __shfl_sync(0xffffffffu, at_row, ((i0 + i) * kRowsAtOnce + sub) & 31);
                    next[i] = src >= 0 && i0 < kLanes ? __ldg(reinterpret_cast<const uint4 *>(a.q + (int64_t)src * D) + piece)
                                                      : make_uint4(0, 0, 0, 0);
                }
            };
            load(0);
#pragma unroll 1
            for (int i0 = 0; i0 < kLanes; i0 += 4) {
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = next[i];
                load(i0 + 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(tile_piece((i0 + i) * kRowsAtOnce + sub, piece)) = v[i];
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&q_full));
            const int pos = p.r.len - p.r.n + (p.g.rowbase + min(rr, p.g.nrows - 1)) / a.G;
            const bool used = mt == 0 || p.g.nrows > kM;
            float ref = 0.0f, pass = -INFINITY, sum = 0.0f;
            uint32_t nans = 0;   // channel blocks that are NaN for this row
            for (int c = p.c0; c < p.c1; ++c, ++tiles) {
                if (!used) continue;
                const uint32_t in = tiles % kInfos;
                ok = wait(info_full[in], (tiles / kInfos) & 1) && wait(s_full[mt], mine & 1);
                ++mine;
                if (!ok) break;
                tc_fence_after();
                const Info info = s_info[in];
                const int t0 = p.g.lo + c * kTok;
                const bool edge = t0 + kTok - 1 > p.g.pos_lo || (a.window && t0 <= p.g.pos_hi - a.window) || info.bad;
                const int upto = pos - t0, from = a.window ? pos - a.window - t0 : -1;   // columns from < i <= upto
                float shrink = 1.0f;   // what O is to be multiplied by before this tile
                F2 part[2] = {0ull, 0ull};
                int q0 = 0;   // the first 32 columns to be taken here
                if (info.bf16) {
                    const RowState st = two_bf16(ts, upto, from, info.bad, a.scale_log2, {ref, pass, sum, shrink});
                    ref = st.ref, pass = st.pass, sum = st.sum, shrink = st.shrink;
                    q0 = kTok / 32;
                }
                // 32 columns at a time (a small loop: unrolled, its code did not stay in the
                // instruction cache): their P takes the place of S that has been read.
                uint32_t r[2][16];
                tmem_ld16(ts, r[0]);
                tmem_ld16(ts + 16, r[1]);
                // scores of 32 columns from r, past m, hidden ones at minus infinity
                auto scores = [&](int q, float (&x)[32]) {
                    const F2 xs2 = pack2(__float_as_uint(a.scale_log2), __float_as_uint(a.scale_log2));
                    const F2 ref2 = pack2(__float_as_uint(-ref), __float_as_uint(-ref));
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const F2 v = fma2(pack2(r[i >> 4][i & 15], r[i >> 4][(i & 15) + 1]), xs2, ref2);
                        x[i] = __uint_as_float((uint32_t)v), x[i + 1] = __uint_as_float((uint32_t)(v >> 32));
                    }
                    if (edge) {
                        const int hi = upto - 32 * q, lo = from - 32 * q;
                        const uint32_t bad = (info.bad >> 2 * q & 1u ? 0xffffu : 0u) | (info.bad >> 2 * q & 2u ? 0xffff0000u : 0u);
                        // bit i: column i is seen
                        uint32_t seen = hi < 0 ? 0u : hi >= 31 ? 0xffffffffu : (2u << hi) - 1u;
                        if (lo >= 0) seen &= lo >= 31 ? 0u : ~((2u << lo) - 1u);
                        seen &= ~bad;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(seen >> i & 1u)) x[i] = -INFINITY;
                    }
                };
                auto largest = [](const float (&x)[32]) {
                    float t4[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) t4[i] = fmaxf(x[i], x[i + 4]);
#pragma unroll
                    for (int i = 8; i < 32; i += 8)
#pragma unroll
                        for (int z = 0; z < 4; ++z) t4[z] = fmaxf(t4[z], fmaxf(x[i + z], x[i + z + 4]));
                    return fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                };
#pragma unroll 1
                for (int q = q0; q < kTok / 32; ++q) {
                    float x[32];
                    uint32_t pk[16];
                    tmem_wait_ld(r[0]);
                    tmem_wait_ld(r[1]);
                    scores(q, x);
                    if (q + 1 < kTok / 32) {
                        tmem_ld16(ts + 32 * q + 32, r[0]);
                        tmem_ld16(ts + 32 * q + 48, r[1]);
                    }
                    // exponentials first: whether m has to rise is known while they are formed
                    const float top = largest(x);
                    F2 more[2] = {0ull, 0ull};
                    auto exponentials = [&]() {
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            x[i] = ex2(x[i]);
                            x[i + 1] = ex2(x[i + 1]);
                            more[i >> 1 & 1] = add2(more[i >> 1 & 1], pack2(__float_as_uint(x[i]), __float_as_uint(x[i + 1])));
                            pk[i / 2] = half2_bits(x[i], x[i + 1]);
                        }
                    };
                    exponentials();
                    if (__any_sync(0xffffffffu, top > pass)) {
                        // m rises by whole powers of two, so that what is scaled stays exact
                        // before there is an m there is nothing to scale
                        const bool none = pass == -INFINITY;
                        const float rise = top == -INFINITY ? 0.0f : none ? ceilf(top) - kRest : fmaxf(ceilf(top) - kRest, 0.0f);
                        if (top != -INFINITY) pass = kAttnTop;
                        ref += rise;
                        const float f = none ? 1.0f : ex2(-rise);
                        sum *= f;
                        shrink *= f;
#pragma unroll
                        for (int i = 0; i < 2; ++i) part[i] = mul2(part[i], pack2(__float_as_uint(f), __float_as_uint(f)));
                        tmem_wait_st();
                        // P so far times f, at most 2^-14 at a time (fp16 has no 2^-25); below 2^-42 nothing is left
                        float left = f;
#pragma unroll 1
                        for (int times = 0; times < 3; ++times) {
                            const float part16 = fmaxf(left, 0x1p-14f);
                            const uint32_t f2 = half2_bits(part16, part16);
#pragma unroll 1
                            for (int z = 0; z < 2 * q; ++z) {
                                uint32_t y[8];
                                tmem_get8(ts + 8 * z, y);
#pragma unroll
                                for (int i = 0; i < 8; ++i) y[i] = mul_half2(y[i], f2);
                                tmem_st8(ts + 8 * z, y);
                            }
                            if (!__any_sync(0xffffffffu, left < 0x1p-14f)) break;
                            tmem_wait_st();
                            left = left < 0x1p-14f ? left * 0x1p14f : 1.0f;
                        }
                        // these columns again, and the next ones' loads
                        tmem_ld16(ts + 32 * q, r[0]);
                        tmem_ld16(ts + 32 * q + 16, r[1]);
                        tmem_wait_ld(r[0]);
                        tmem_wait_ld(r[1]);
                        scores(q, x);
                        more[0] = more[1] = 0ull;
                        exponentials();
                        if (q + 1 < kTok / 32) {
                            tmem_ld16(ts + 32 * q + 32, r[0]);
                            tmem_ld16(ts + 32 * q + 48, r[1]);
                        }
                    }
                    part[0] = add2(part[0], more[0]);
                    part[1] = add2(part[1], more[1]);
                    tmem_st16(ts + 16 * q, pk);
                }
                tmem_wait_ld(r[0]);   // (where the loop took none)
                tmem_wait_ld(r[1]);
                part[0] = add2(part[0], part[1]);
                sum += __uint_as_float((uint32_t)part[0]) + __uint_as_float((uint32_t)(part[0] >> 32));
                if (c > p.c0 && __any_sync(0xffffffffu, shrink != 1.0f)) {   // S was there: the products before it are done
#pragma unroll 1
                    for (int q = 0; q < D / 16; ++q) {
                        uint32_t r[16];
                        tmem_ld16(to + 16 * q, r);
                        tmem_wait_ld(r);
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * shrink);
                        tmem_st16(to + 16 * q, r);
                    }
                }
                tmem_wait_st();
                if (info.nan) {
#pragma unroll 1
                    for (int t = 0; t < kTok; t += 2) {   // (not by P, which fp16 may have made zero)
                        const uint2 n8 = s_nan[in][t / 2];
                        const bool there = !(info.bad >> (t >> 4) & 1u);
                        if (there && t <= upto && t > from) nans |= n8.x;
                        if (there && t + 1 <= upto && t + 1 > from) nans |= n8.y;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&p_ready[mt]));
            }
            ok = ok && wait(o_full, pieces & 1);
            ++pieces;
            if (!ok) break;
            tc_fence_after();
            const bool whole = p.c0 == 0 && p.c1 == p.g.tiles;
            if (tid == 0 && p.c0 == 0 && !whole) {   // the CTA's last piece: units to come are those after walk.u
                const AttnCut cut = {p.r.row0, p.h * a.G, p.g.rowbase, p.g.nrows,
                                     (int)((walk.u + (p.g.tiles - p.c1) - 1) / per), {}};
                a.cuts[blockIdx.x] = cut;
            }
            float *dst = a.part + (int64_t)(2 * blockIdx.x + (p.c0 == 0)) * kWideRows * (D + 2);
            const float inv = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
            if (!whole) dst[kWideRows * D + rr] = pass == -INFINITY ? -INFINITY : ref, dst[kWideRows * (D + 1) + rr] = sum;
            else if (there && a.lse) a.lse[at] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.69314718f;
            if (used) {
                // By way of the queries' place (their products are done), so that rows leave whole; fp32 in
                // two halves.  (A thread to a row: 8000 cycles a piece, 5000 so.)
                const bool f32 = !whole || !a.out_bf16;
                const int cols = f32 ? D / 2 : D;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += cols) {
                    uint32_t r[16];
                    tmem_ld16(to + c0, r);
#pragma unroll 1
                    for (int q = 0; q < cols / 16; ++q) {
                        tmem_wait_ld(r);
                        float x[16];
                        const bool gone = nans >> (8 * ((c0 + 16 * q) / 32)) & 1u;
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = gone ? NAN : inv == 0.0f ? 0.0f : __uint_as_float(r[i]) * inv;
                        if (q + 1 < cols / 16) tmem_ld16(to + c0 + 16 * q + 16, r);
                        if (f32) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                *reinterpret_cast<float4 *>(tile_piece(lane, 4 * q + i)) =
                                    make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                        } else {
                            uint32_t y[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                                y[i] = *reinterpret_cast<const uint32_t *>(&b2);
                            }
                            *reinterpret_cast<uint4 *>(tile_piece(lane, 2 * q)) = make_uint4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<uint4 *>(tile_piece(lane, 2 * q + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
                        }
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int i = 0; i < kLanes; ++i) {
                        const int r = i * kRowsAtOnce + sub, src = __shfl_sync(0xffffffffu, at_row, r);
                        if (src < 0) continue;
                        const uint4 v = *reinterpret_cast<const uint4 *>(tile_piece(r, piece));
                        uint4 *to_row = !whole  ? reinterpret_cast<uint4 *>(dst + (int64_t)(rr - lane + r) * D + c0)
                                        : f32 ? reinterpret_cast<uint4 *>(static_cast<float *>(a.out) + (int64_t)src * D + c0)
                                              : reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + (int64_t)src * D);
                        to_row[piece] = v;
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();   // O may be written again once the next query is there
        }
    } else if (warp < kMmaWarp) {
        // ---- keys and values into shared memory -------------------------------------------
        // A lane takes 16-byte pieces of codes (32 channels, one scale): eight
        // neighbouring lanes the same piece of eight tokens, so that stores meet no
        // bank twice; a warp's 32 tokens in `I` rounds.
        constexpr int kIn = D / 32, I = kIn, kRoundRows = 32 / kIn;
        const int dw = warp - kSoftWarps;
        const int pc = D == 128 ? lane >> 3 : lane >> 3 & 1;
        const int pr = D == 128 ? lane & 7 : (lane & 7) + (lane >> 4) * 8;
        const int64_t kv_rows = (int64_t)a.Hk << a.page_shift;
        const int in_page = (1 << a.page_shift) - 1;
        while (ok && walk.next(w, entries, p)) {
            if (p.c0 == p.c1) continue;
            const int32_t *table = a.table + (int64_t)p.b * a.max_pages;
            // What the next tile needs is on its way: pages two tiles ahead, scales one, keys
            // from when this tile's have been taken; values from the tile's own start.  (Loads
            // issued before older ones are used were waited for with them.)
            uint4 kc[I], vc[I];
            uint32_t kb[I], vb[I];   // scale bytes of this tile; 0 where there is nothing
            uint32_t kn[I], vn[I];   // of the next
            int64_t rows[2];         // of the next tile's keys for each 16 tokens: this lane's first; below 0: nothing
            int ids[2];              // pages of the tile behind it; -1: none, kHidden: nothing to see
            constexpr int kHidden = INT_MIN;
            auto load_ids = [&](int c) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = p.g.lo + c * kTok + 32 * dw + 16 * i;
                    // (an id below zero is not kHidden, whatever it is)
                    ids[i] = c < p.c1 && t <= p.g.pos_hi ? max(__ldg(table + (t >> a.page_shift)), -1) : kHidden;
                }
            };
            // rounds of 16 / kRoundRows for each 16 tokens
            constexpr int kRounds = 16 / kRoundRows;
            auto load_codes = [&](uint4 (&x)[I], int64_t rows_on) {
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    const int64_t r = rows[i / kRounds];
                    x[i] = r >= 0 ? __ldg(reinterpret_cast<const uint4 *>(a.codes + (r + rows_on) * (D / 2)) + pc +
                                          (i % kRounds) * kRoundRows * (D / 32))
                                  : make_uint4(0, 0, 0, 0);
                }
            };
            uint32_t next_lost = 0;   // bit i: tokens 16 i .. of the next tile have no page
            int next_seen = 0;        // its tokens that rows see
            // From the pages of tile c: its rows, and its scales on their way.
            auto load_scales = [&](int c) {
                next_lost = 0;
                const int t0 = p.g.lo + c * kTok;
                next_seen = p.g.pos_hi + 1 - t0;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    rows[g] = -1;
                    if (ids[g] >= 0 && ids[g] < a.pages) {
                        rows[g] = (((int64_t)ids[g] * 2 * a.Hk + p.h) << a.page_shift) + ((t0 + 32 * dw + 16 * g + pr) & in_page);
                    } else if (ids[g] != kHidden) {
                        next_lost |= 1u << (2 * dw + g);
                        if (a.status && lane == 0) atomicOr(a.status, MOE_DEV_BAD_INDEX);
                    }
                }
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    kn[i] = vn[i] = 0;
                    const int64_t r = rows[i / kRounds];
                    if (r < 0) continue;
                    const uint8_t *s = a.scales + r * kBlocks + pc + (i % kRounds) * kRoundRows * kBlocks;
                    kn[i] = __ldg(s);
                    vn[i] = __ldg(s + kv_rows * kBlocks);
                }
            };
            load_ids(p.c0);
            load_scales(p.c0);
            load_ids(p.c0 + 1);
            load_codes(kc, 0);
            for (int c = p.c0; c < p.c1; ++c, ++tiles) {
                const uint32_t stage = tiles % kStages, in = tiles % kInfos;
                uint32_t bad = next_lost, nan = 0, far = 0, odd = 0;   // of all the warp's tokens
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    // rows behind the last token may hold anything
                    const bool seen = 32 * dw + kRoundRows * i + pr < next_seen;
                    kb[i] = seen ? kn[i] : 0u, vb[i] = seen ? vn[i] : 0u;
                    far |= kb[i] > 142u;
                    nan |= vb[i] == 255u;
                    odd |= seen && vb[i] - kLeastHalf > kMostHalf - kLeastHalf && vb[i] != 255u;
                }
                nan = __any_sync(0xffffffffu, nan);
                far = __any_sync(0xffffffffu, far);
                odd = __any_sync(0xffffffffu, odd);
                if (lane == 0) {
                    s_e[tiles & 1][dw] = make_uint4(bad, nan, odd, 0);
                    mbar_arrive(smem_u32(&e_full[tiles & 1]));
                }
                load_codes(vc, kv_rows);
                load_scales(c + 1);
                load_ids(c + 2);
                ok = wait(e_full[tiles & 1], (tiles >> 1) & 1);
                if (!ok) break;
#pragma unroll
                for (int x = 0; x < kUnpackWarps; ++x) {
                    const uint4 e = s_e[tiles & 1][x];
                    bad |= e.x, nan |= e.y, odd |= e.z;
                }
                ok = wait(k_empty[stage], ((tiles / kStages) & 1) ^ 1u);
                if (!ok) break;
                if (dw == 0 && lane == 0) {
                    Info info;
                    info.bad = bad, info.nan = nan, info.bf16 = odd;
                    s_info[in] = info;
                }
                if (nan)
#pragma unroll
                    for (int i = 0; i < I; ++i) {
                        const int t = 32 * dw + kRoundRows * i + pr;
                        uint8_t *n = reinterpret_cast<uint8_t *>(s_nan[in]) + 4 * t + pc;
                        n[0] = vb[i] == 255u;
                        if (kIn == 2) n[2] = 0;
                    }
                // codes of 32 channels (a lane's 16 bytes) of token t to shared memory, by `to16` of pairs
                auto widen = [&](const uint4 &codes, uint8_t *dst, int t, auto to16) {
                    const uint32_t x[4] = {codes.x, codes.y, codes.z, codes.w};
                    uint8_t *rowp = dst + (pc >> 1) * S::kHalf + t * 128;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t hv[4];
                        mx4_half8(x[j], hv);
                        *reinterpret_cast<uint4 *>(rowp + ((((pc & 1) * 4 + j) ^ (t & 7)) << 4)) =
                            make_uint4(to16(hv[0]), to16(hv[1]), to16(hv[2]), to16(hv[3]));
                    }
                };
                // where piece i of this lane's is, and what a scale has beyond bf16's one factor
                auto piece_at = [&](uint8_t *dst, int i) {
                    const int t = 32 * dw + kRoundRows * (i >> 2) + pr;
                    return reinterpret_cast<uint4 *>(dst + (pc >> 1) * S::kHalf + t * 128 + ((((pc & 1) * 4 + (i & 3)) ^ (t & 7)) << 4));
                };
                auto beyond = [](uint32_t byte) { return ((127u + max((int)byte - 142, 0)) << 7) * 0x10001u; };
                // Keys: bf16, 2^(e - 127) by way of 2^-112 and 2^(e - 15); from 2^16 on that passes bf16's
                // largest and is made of two
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    uint8_t *const dst = smem + S::kK + stage * S::kTileBytes;
                    const int t = 32 * dw + kRoundRows * i + pr;
                    const uint32_t f = (kb[i] == 255u ? 0x7fc0u : min(kb[i] + 112u, 254u) << 7) * 0x10001u;
                    widen(kc[i], dst, t, [&](uint32_t h) { return mul_bf162(bf16_of_half2(h), f); });
                }
                if (far)   // (its own small loop: in line, it would be in the instruction cache's way)
#pragma unroll 1
                    for (int i = 0; i < 4 * I; ++i) {
                        const uint32_t g = beyond(i < 4 ? kb[0] : i < 8 ? kb[1] : i < 12 ? kb[2 % I] : kb[3 % I]);
                        uint4 *const at = piece_at(smem + S::kK + stage * S::kTileBytes, i);
                        const uint4 y = *at;
                        *at = make_uint4(mul_bf162(y.x, g), mul_bf162(y.y, g), mul_bf162(y.z, g), mul_bf162(y.w, g));
                    }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&info_full[in]));
                    mbar_arrive(smem_u32(&k_full[stage]));
                }
                load_codes(kc, 0);
                ok = wait(v_empty[stage], ((tiles / kStages) & 1) ^ 1u);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < I; ++i)
                {   // values: fp16 times 2^(e - 127), or unscaled where the tile's are bf16
                    const uint32_t f = odd ? 0x3c003c00u : vb[i] == 255u ? 0u : half2_bits(__uint_as_float(vb[i] << 23), __uint_as_float(vb[i] << 23));
                    widen(vc[i], smem + S::kV + stage * S::kTileBytes, 32 * dw + kRoundRows * i + pr,
                          [&](uint32_t h) { return mul_half2(h, f); });
                }
                if (odd)   // to bf16, as keys
#pragma unroll 1
                    for (int i = 0; i < 4 * I; ++i) {
                        const uint32_t byte = i < 4 ? vb[0] : i < 8 ? vb[1] : i < 12 ? vb[2 % I] : vb[3 % I];
                        const uint32_t f = byte == 255u ? 0u : (min(byte + 112u, 254u) << 7) * 0x10001u, g = beyond(byte);
                        uint4 *const at = piece_at(smem + S::kV + stage * S::kTileBytes, i);
                        const uint4 y = *at;
                        auto to16 = [&](uint32_t h) { return mul_bf162(mul_bf162(bf16_of_half2(h), f), g); };
                        *at = make_uint4(to16(y.x), to16(y.y), to16(y.z), to16(y.w));
                    }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&v_full[stage]));
            }
        }
    } else {
        // ---- products ---------------------------------------------------------------------
        const bool elected = elect_one();
        constexpr uint32_t kQK = idesc_bf16(kM, kTok), kPV = idesc_mn(kM, D, false), kPV2 = idesc_mn(kM, D, true);
        uint32_t made[2] = {0, 0};   // P of each half that products have taken
        while (ok && walk.next(w, entries, p)) {
            if (p.c0 == p.c1) continue;
            const int n = p.c1 - p.c0, halves = p.g.nrows > kM ? 2 : 1;
            auto qk = [&](int mt, uint32_t tile) {
                const uint32_t stage = tile % kStages;
                if (elected) {
                    const uint64_t q = sdesc_k_sw128(base + S::kQ + mt * S::kTileBytes);
                    const uint64_t k = sdesc_k_sw128(base + S::kK + stage * S::kTileBytes);
#pragma unroll
                    for (int s = 0; s < D / 16; ++s) {
                        const uint32_t off = (s >> 2) * (S::kHalf >> 4) + (s & 3) * 2;
                        mma_f16(tmem + mt * kTok, q + off, k + off, kQK, s > 0);
                    }
                    mma_commit(smem_u32(&s_full[mt]));
                    if (mt == halves - 1) mma_commit(smem_u32(&k_empty[stage]));
                }
                __syncwarp();
            };
            auto have_keys = [&](uint32_t tile) {
                const bool good = wait(k_full[tile % kStages], (tile / kStages) & 1);
                tc_fence_after();
                return good;
            };
            ok = wait(q_full, pieces & 1) && have_keys(tiles);
            ++pieces;
            if (!ok) break;
            for (int mt = 0; mt < halves; ++mt) qk(mt, tiles);
            for (int j = 0; j < n && ok; ++j, ++tiles) {
                const uint32_t stage = tiles % kStages;
                ok = wait(v_full[stage], (tiles / kStages) & 1);
                for (int mt = 0; mt < halves && ok; ++mt) {
                    ok = wait(p_ready[mt], made[mt] & 1);
                    ++made[mt];
                    if (!ok) break;
                    tc_fence_after();
                    if (elected) {
                        const uint64_t v = sdesc_mn_sw128(base + S::kV + stage * S::kTileBytes);
                        const uint32_t p16 = tmem + mt * kTok, o = tmem + S::kO + mt * D;
                        if (!s_info[tiles % kInfos].bf16) {
#pragma unroll
                            for (int s = 0; s < kTok / 16; ++s)
                                mma_f16_ta(o, p16 + 8 * s, v + s * (2048 >> 4), kPV, j > 0 || s > 0);
                        } else {
#pragma unroll 1
                            for (int s = 0; s < kTok / 16; ++s) {
                                const uint32_t at = p16 + 16 * s;
                                mma_f16_ta(o, at, v + s * (2048 >> 4), kPV2, j > 0 || s > 0);
                                mma_f16_ta(o, at + 8, v + s * (2048 >> 4), kPV2, 1);
                            }
                        }
                        if (mt == halves - 1) mma_commit(smem_u32(&v_empty[stage]));
                    }
                    __syncwarp();
                    if (j + 1 < n) {   // into S that these products have taken P from
                        if (mt == 0) ok = have_keys(tiles + 1);
                        if (ok) qk(mt, tiles + 1);
                    }
                }
            }
            if (elected && ok) mma_commit(smem_u32(&o_full));
            __syncwarp();
        }
        if (elected) {
            mma_commit(smem_u32(&drain_bar));
            wait_drain(smem_u32(&drain_bar), 0);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

int entries_bound(const moe_cache_attn *d, int G) {
    return (int)std::min<int64_t>((int64_t)d->rows * G / kWideRows + std::min(d->requests, d->rows), 1 << 30);
}

struct WideLayout {
    size_t units, per, request, first, cuts, part, total;
};
WideLayout wide_layout(const moe_cache_attn *d, const moe_cache4 *cache) {
    WideLayout l;
    const size_t e = (size_t)entries_bound(d, d->q_heads / cache->kv_heads);
    l.units = 0;
    l.per = align_up(8 * (e + 1));
    l.request = l.per + align_up(8);
    l.first = l.request + align_up(4 * e);
    l.cuts = l.first + align_up(4 * ((size_t)d->requests + 1));
    l.part = l.cuts + align_up(sizeof(AttnCut) * sm_count());
    l.total = l.part + align_up(sizeof(float) * 2 * (size_t)sm_count() * kWideRows * (cache->dim + 2));
    return l;
}

template <int D>
int launch(const WideArgs &w, cudaStream_t s) {
    const int ctas = sm_count();
    MOE_CUDA_TRY(cudaFuncSetAttribute(attention4_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      WideShape<D>::kSmem));
    if (int rc = launch_dependent(wide_plan_kernel, dim3(1), dim3(1024), 0, s, (const WideArgs)w, ctas)) return rc;
    if (int rc = launch_dependent(attention4_wide_kernel<D>, dim3((unsigned)ctas), dim3(kWideThreads),
                                  WideShape<D>::kSmem, s, (const WideArgs)w))
        return rc;
    return launch_attention4_join(w.a, D, kWideRows, ctas, s);
}

}  // namespace

size_t attention4_wide_workspace(const moe_cache_attn *d, const moe_cache4 *cache) {
    return wide_layout(d, cache).total;
}

int launch_attention4_wide(const AttnArgs &args, const moe_cache_attn *d, const moe_cache4 *cache, int few_rows,
                           void *ws, cudaStream_t s) {
    const WideLayout l = wide_layout(d, cache);
    uint8_t *p = static_cast<uint8_t *>(ws);
    WideArgs w;
    w.a = args;
    w.a.part = reinterpret_cast<float *>(p + l.part);
    w.a.cuts = reinterpret_cast<AttnCut *>(p + l.cuts);
    w.few_rows = few_rows;
    w.max_entries = entries_bound(d, args.G);
    w.units = reinterpret_cast<int64_t *>(p + l.units);
    w.per = reinterpret_cast<int64_t *>(p + l.per);
    w.entry_request = reinterpret_cast<int32_t *>(p + l.request);
    w.first_entry = reinterpret_cast<int32_t *>(p + l.first);
    return cache->dim == 64 ? launch<64>(w, s) : launch<128>(w, s);
}

}  // namespace moe
