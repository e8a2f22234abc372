// Grouped products of MXFP4 rows and weights:
//   C[r, n] = sum_k A[r, k] W[g, n, k]      (rows r of group g)
// on the tensor cores' block-scaled four-bit kind (tcgen05.mma kind::mxf4:
// e2m1 operands, one power-of-two scale for 32 of K, fp32 accumulation in
// tensor memory), with a plain epilogue (fp32 or bf16 C) or SwiGLU and the
// MXFP4 quantisation of h (gate block and up block of the same 128 features
// in one tile).
//
// Persistent CTAs, one to an SM, take tiles of 256 weight rows (N, two blocks
// of 128) and 128 token rows (M), or, in pairs of CTAs (tcgen05 cta_group::2,
// clusters of two), 256 token rows: each CTA of a pair loads its own 128 token
// rows and one of the two weight blocks, and the products read both CTAs'
// shared memory, which takes a third off what an SM has to load for a product.
// A stage of the ring holds 256 of K: the token rows' codes (TMA boxes of 128
// bytes a row, 128-byte swizzle), the weight tiles (bulk copies, stored
// pre-swizzled), the weights' scale bytes (stored in the order tensor memory
// wants), and the token rows' scale bytes, which come row-major from global
// memory and are put in that order: a warp's lane L holds rows L, L+32, L+64,
// L+96, whose four words of four scales are one 16-byte chunk, to be repeated
// in the four lane quarters.
//
// Between the CTAs of a pair: the first CTA's products wait for both CTAs'
// scale warps (sf_bar) and epilogues (acc_empty), whose arrivals on the other
// CTA's barrier have the default CTA scope, with which the memory model does
// not order memory between CTAs.  What stands behind them needs no more:
// copies into shared memory that have arrived on their own barrier, stores to
// and loads from tensor memory that tcgen05.wait has waited for. All of it has
// been performed before the arrival is issued, and nothing that a thread of one
// CTA stores itself is read by the other (the token rows' scale bytes are
// put into shared memory for the CTA's own warps).  Releases at cluster scope
// were 127 -> 295 us for 8192 x 7168 x 7168.  The products' own arrivals on
// both CTAs' barriers are the tensor core's (multicast commit).
//
// What bounds it: weights read once for few rows (254 MB of down products for
// 273 rows in 39 us, 95% of the copy rate); for many, products and the way from
// one tile to the next, since the accumulator and the scales leave no room in
// tensor memory for a second accumulator: 8192 x 7168 x 7168 takes 116 us, 7.3
// PFLOP/s, of which about 640 cycles a stage in products and 2000 a tile where
// they wait for the epilogue to read it.  fp32 C, twice the bytes to store, on
// one GPU with bf16 C beside it: 273 rows 38.3 / 37.6 us, 16411 rows of K 2048 in
// 8 groups 129 / 99 (80 at the copy rate), 8192 x 7168 x 7168 133 / 116.
// On the way there, same product: 267 us -> 253 waits that let the hardware
// hold the thread; -> 234 one copy for both K blocks' scale bytes; -> 199 a
// warp for each ring slot to issue its copies; -> 176 scales stored to tensor
// memory by warps instead of tcgen05.cp; -> 164 one elected thread issues, with
// addresses formed before the slot is free; -> 127 pairs; -> 124 two slots to
// an operand warp (more registers for the epilogue); -> 121 stores past L1; ->
// 116 weights that are read again stay in L2.
//
// The hardware applies the scales, so nothing is promoted on the way and an
// accumulator runs over all of K; the epilogue sees each output once.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "internal.h"
#include "mx4.cuh"
#include "numerics.cuh"
#include "ptx.cuh"
#include "tma_host.h"

namespace moe {
namespace {

constexpr int kTN = 256;               // columns of a tile: two weight blocks
constexpr int kTileBytes = 128 * 64;   // 128 rows x 128 of K
constexpr int kMaxGroups = 1024;
constexpr int kTmemCols = 512, kSfCol = kTN, kSfStage = 2 * (4 + 8);

// A ring slot: 128 token rows x 256 of K (this CTA's), then the weights of both
// blocks ([K block][weight block]) or, in a pair, of this CTA's one; the scales
// of the token rows and of both weight blocks ([weight block][K block]), 512
// bytes for a block of 128 rows and of K.
// Tensor memory: the accumulator, then for each slot and K block the scales of
// the token rows (4 columns) and of the weight rows (8).
template <bool SW, bool PAIR>
struct Shape {
    static constexpr int kTM = PAIR ? 256 : 128;   // token rows of a tile
    static constexpr int kBlocks = PAIR ? 1 : 2;   // weight blocks in a CTA's ring
    static constexpr int kStages = PAIR ? 6 : 4;
    static constexpr int kAOff = 0, kBOff = 2 * kTileBytes;
    static constexpr int kSAOff = kBOff + 2 * kBlocks * kTileBytes, kSBOff = kSAOff + 2 * 512;
    static constexpr int kStageBytes = kSBOff + 4 * 512;
    static constexpr int kSmemBytes = kStages * kStageBytes + 1024;
    static constexpr int kMmaWarp = 0, kFirstSlotWarp = 1, kSlotWarps = kStages / 2;   // two slots each
    static constexpr int kFirstSfWarp = kFirstSlotWarp + kSlotWarps, kSfWarps = 4;
    static constexpr int kFirstEpiWarp = kFirstSfWarp + kSfWarps, kEpiWarps = SW ? 16 : 8;
    static constexpr int kThreads = (kFirstEpiWarp + kEpiWarps) * 32;
    static_assert(kSfCol + kStages * kSfStage <= kTmemCols, "tensor memory");
};

struct Mx4Args {
    int groups, n_out, k_dim, rows;
    const uint8_t *a_scales;   // [rows, k_dim / 32]
    const int32_t *offsets;
    const uint8_t *w, *w_scales;
    void *c;                   // plain: [rows, n_out]; SwiGLU: codes [rows, n_out / 4]
    uint8_t *h_scales;         // SwiGLU: [rows, n_out / 64]
    int c_bf16;
    int32_t *status;
};

// instruction descriptor: e2m1 x e2m1, ue8m0 scales, K = 64, scale bytes `sf`
// and `sf` + 1 of each 32-bit column
__host__ __device__ constexpr uint32_t idesc_mxf4(int rows, int sf) {
    return ((uint32_t)sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kTN >> 3) << 17) | (1u << 23) |
           ((uint32_t)(rows >> 4) << 24) | ((uint32_t)sf << 29);
}

struct Tile {
    int g, nt, row0, nvalid;
};

// Tile t -> (group, column tile; this CTA's first row and its valid rows, of the
// second CTA possibly none); s_tiles holds each group's first tile.  Row tiles
// of one column tile are neighbours, so they share its weights in L2.
template <int kTM>
__device__ __forceinline__ Tile decode(int t, int rank, int G, const int *s_tiles, const int *s_off) {
    int lo = 0, hi = G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tiles[mid] <= t) lo = mid;
        else hi = mid;
    }
    Tile w;
    w.g = lo;
    const int rows = s_off[lo + 1] - s_off[lo], mtiles = (rows + kTM - 1) / kTM;
    const int local = t - s_tiles[lo];
    w.nt = local / mtiles;
    const int mt = local - w.nt * mtiles;
    const int r = mt * kTM + rank * 128;
    w.row0 = s_off[lo] + r;
    w.nvalid = max(0, min(128, rows - r));
    return w;
}

// 32 bytes, one sector, in one store, without a line in L1 (16411 rows of K 2048:
// 110 us with, 100 without)
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

template <bool SW, bool PAIR>
__global__ void __launch_bounds__((Shape<SW, PAIR>::kThreads), 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                    const Mx4Args args) {
    using namespace ptx;
    using S = Shape<SW, PAIR>;
    constexpr int kTM = S::kTM, kStages = S::kStages, kStageBytes = S::kStageBytes, kThreads = S::kThreads;
    constexpr int kAOff = S::kAOff, kBOff = S::kBOff, kSAOff = S::kSAOff, kSBOff = S::kSBOff;
    constexpr int kMmaWarp = S::kMmaWarp, kFirstSlotWarp = S::kFirstSlotWarp, kFirstSfWarp = S::kFirstSfWarp;
    constexpr int kFirstEpiWarp = S::kFirstEpiWarp, kCtas = PAIR ? 2 : 1;
    extern __shared__ uint8_t dsmem[];
    __shared__ __align__(8) uint64_t full_bar[kStages], sf_bar[kStages], empty_bar[kStages], acc_full, acc_empty, drain_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_abort, s_bad;
    __shared__ int s_off[kMaxGroups + 1], s_tiles[kMaxGroups + 1];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t smem_base = (smem_u32(dsmem) + 1023u) & ~1023u;
    const int rank = PAIR ? (int)cluster_rank() : 0, pair = blockIdx.x / kCtas, pairs = gridDim.x / kCtas;
    const int G = args.groups;
    const int nblocks = args.n_out / 128;                       // weight blocks of a group
    const int NT = SW ? nblocks / 2 : (nblocks + 1) / 2;        // column tiles
    const int KB = args.k_dim / 128, steps = (KB + 1) / 2;      // K blocks; ring stages a tile
    volatile int *abort_flag = &s_abort;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&sf_bar[s]), kCtas * S::kSfWarps);   // of a pair, in its first CTA
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
        mbar_init(smem_u32(&acc_full), 1);
        mbar_init(smem_u32(&acc_empty), kCtas * S::kEpiWarps);     // as sf_bar
        mbar_init(smem_u32(&drain_bar), 1);
        s_abort = 0;
        s_bad = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        if constexpr (PAIR) {
            tmem_alloc2(smem_u32(&tmem_slot), kTmemCols);
            tmem_relinquish2();
        } else {
            tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
            tmem_relinquish();
        }
    }
    if (warp == kFirstSlotWarp && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmA32);
    }
    pdl_launch_dependents();
    pdl_wait();
    for (int i = threadIdx.x; i <= G; i += kThreads) s_off[i] = args.offsets[i];
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += kThreads) {
        const int a = s_off[g], b = s_off[g + 1];
        if (a < 0 || b < a || b > args.rows) s_bad = 1;
    }
    __syncthreads();
    auto tiles_of = [&](int g) { return NT * ((s_off[g + 1] - s_off[g] + kTM - 1) / kTM); };
    if (warp == 0 && !s_bad) {   // prefix over groups: lane L owns a contiguous run
        const int per = (G + 31) / 32, g0 = lane * per;
        int local = 0;
        for (int q = 0; q < per; ++q)
            if (g0 + q < G) local += tiles_of(g0 + q);
        int incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += n;
        }
        int run = incl - local;
        for (int q = 0; q < per; ++q)
            if (g0 + q < G) {
                s_tiles[g0 + q] = run;
                run += tiles_of(g0 + q);
            }
        if (lane == 31) s_tiles[G] = incl;
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();   // both CTAs' barriers are set up
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int total = s_bad ? 0 : s_tiles[G];
    if (s_bad && threadIdx.x == 0 && blockIdx.x == 0 && args.status)
        atomicOr(args.status, MOE_DEV_BAD_OFFSETS);

    if (warp == kMmaWarp) {
        // ---- products, of both CTAs by the first ---------------------------------------
        // The whole warp waits and one thread issues.
        const bool elected = elect_one();
        auto commit = [](uint32_t bar, uint16_t ctas) {
            if constexpr (PAIR) mma_commit2(bar, ctas);
            else mma_commit(bar);
        };
        uint32_t it = 0, tiles = 0;
        bool ok = true;
        for (int t = pair; t < total && ok && rank == 0; t += pairs, ++tiles) {
            ok = wait_bounded(smem_u32(&acc_empty), (tiles & 1) ^ 1u, abort_flag, args.status,
                              MOE_DEV_TIMEOUT);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            for (int s = 0; s < steps; ++s, ++it) {
                const uint32_t slot = it % kStages;
                ok = wait_bounded(smem_u32(&sf_bar[slot]), (it / kStages) & 1, abort_flag, args.status,
                                        MOE_DEV_TIMEOUT);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t base = smem_base + slot * kStageBytes;
                const uint32_t sf = tmem + kSfCol + slot * kSfStage;
                if (elected) {
                    const uint64_t ad = sdesc_k_sw128(base + kAOff), bd = sdesc_k_sw64(base + kBOff);
                    constexpr int kNext = S::kBlocks * kTileBytes / 16;   // the next K block's weights
                    auto product = [&](uint64_t a, uint64_t b, uint32_t idesc, uint32_t scales, uint32_t add) {
                        if constexpr (PAIR) mma2_mxf4(tmem, a, b, idesc, scales, scales + 4, add);
                        else mma_mxf4(tmem, a, b, idesc, scales, scales + 4, add);
                    };
                    product(ad, bd, idesc_mxf4(kTM, 0), sf, s > 0);
                    product(ad + 2, bd + 2, idesc_mxf4(kTM, 2), sf, 1);
                    if (2 * s + 1 < KB) {
                        product(ad + 4, bd + kNext, idesc_mxf4(kTM, 0), sf + 12, 1);
                        product(ad + 6, bd + kNext + 2, idesc_mxf4(kTM, 2), sf + 12, 1);
                    }
                    commit(smem_u32(&empty_bar[slot]), 3);
                    if (s == steps - 1) commit(smem_u32(&acc_full), 3);
                }
                __syncwarp();
            }
        }
        if (elected && rank == 0) {
            commit(smem_u32(&drain_bar), 1);
            wait_drain(smem_u32(&drain_bar), 0);
        }
        __syncwarp();
    } else if (warp < kFirstSfWarp) {
        // ---- operands: each of these warps has two of the ring's slots -----------------
        // One thread issues a stage's copies; the warp puts the token rows'
        // scale bytes into their place.  Addresses and scale bytes are there
        // before the slot is free: from the last product of a stage to the next
        // one's in its slot everything here is in line.  (One thread issuing
        // every stage's copies kept the products waiting; with the addresses
        // formed after the wait, by lane 0, a stage's copies took 1240 cycles to
        // issue.)
        const uint32_t mine = warp - kFirstSlotWarp;
        uint8_t *smem = dsmem + (smem_base - smem_u32(dsmem));
        const size_t pitch = args.k_dim / 32;
        const uint64_t pol_once = policy_evict_first(), pol_again = policy_evict_last();
        uint32_t it = mine, first = mine;   // the stage that is next; its step in the tile
        bool ok = true;
        for (int t = pair; t < total && ok; t += pairs) {
            if ((int)first >= steps) {     // none in this tile
                first -= steps;
                continue;
            }
            const Tile tl = decode<kTM>(t, rank, G, s_tiles, s_off);
            const int nb = SW || 2 * tl.nt + 1 < nblocks ? 2 : 1;
            const int copies = PAIR ? rank < nb : nb;                 // weight blocks that this CTA loads
            const bool wide = tl.nvalid > 32, two = tl.nvalid > 64;   // boxes of 64 rows, or one of 32
            const uint32_t abytes = (two ? 128 : wide ? 64 : tl.nvalid ? 32 : 0) * 128;
            const int last = s_off[tl.g + 1] - 1;
            const CUtensorMap *tma = wide ? &tmA : &tmA32;
            const size_t w0 = ((size_t)tl.g * nblocks + (SW ? tl.nt : 2 * tl.nt)) * KB;   // tiles
            const size_t w1 = w0 + (size_t)(SW ? NT : 1) * KB;
            // weights that further row tiles read stay in L2 (8192 x 7168 x 7168:
            // 121 -> 116 us), others make room
            const uint64_t pol_w = s_off[tl.g + 1] - s_off[tl.g] > kTM ? pol_again : pol_once;
            const uint8_t *rows[4];   // this lane's rows' scale bytes
#pragma unroll
            for (int q = 0; q < 4; ++q)
                rows[q] = args.a_scales + (size_t)min(tl.row0 + lane + 32 * q, last) * pitch;
            int s = first;
            for (; s < steps; s += S::kSlotWarps, it += S::kSlotWarps) {
                const uint32_t slot = it % kStages, fb = smem_u32(&full_bar[slot]);
                const uint32_t base = smem_base + slot * kStageBytes;
                const int nk = min(2, KB - 2 * s);
                const uint8_t *wa = args.w + ((rank ? w1 : w0) + 2 * s) * kTileBytes, *wb = args.w + (w1 + 2 * s) * kTileBytes;
                const uint8_t *sa = args.w_scales + (w0 + 2 * s) * 512, *sb = args.w_scales + (w1 + 2 * s) * 512;
                const uint32_t bytes = abytes + nk * (copies * kTileBytes + nb * 512);
                uint32_t v[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int q = 0; q < 4; ++q)   // rows past the last are the last: not stored
                        v[k][q] = __ldg(reinterpret_cast<const uint32_t *>(rows[q] + (2 * s + (k < nk ? k : 0)) * 4));
                ok = wait_bounded(smem_u32(&empty_bar[slot]), ((it / kStages) & 1) ^ 1u, abort_flag, args.status,
                                  MOE_DEV_TIMEOUT);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (elect_one()) {
                    mbar_expect_tx(fb, bytes);
                    if (PAIR) {   // a block's tiles along K are consecutive
                        if (copies) bulk_load(base + kBOff, wa, nk * kTileBytes, fb, pol_w);
                    } else {
                        bulk_load(base + kBOff, wa, kTileBytes, fb, pol_w);
                        if (nb > 1) bulk_load(base + kBOff + kTileBytes, wb, kTileBytes, fb, pol_w);
                        if (nk > 1) {
                            bulk_load(base + kBOff + 2 * kTileBytes, wa + kTileBytes, kTileBytes, fb, pol_w);
                            if (nb > 1) bulk_load(base + kBOff + 3 * kTileBytes, wb + kTileBytes, kTileBytes, fb, pol_w);
                        }
                    }
                    if (tl.nvalid) tma_load_2d(base + kAOff, tma, s * 128, tl.row0, fb, pol_again);
                    if (two) tma_load_2d(base + kAOff + 64 * 128, tma, s * 128, tl.row0 + 64, fb, pol_again);
                    bulk_load(base + kSBOff, sa, nk * 512, fb, pol_w);
                    if (nb > 1) bulk_load(base + kSBOff + 2 * 512, sb, nk * 512, fb, pol_w);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    *reinterpret_cast<uint4 *>(smem + slot * kStageBytes + kSAOff + k * 512 + lane * 16) =
                        make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
                __syncwarp();
                if (elect_one()) mbar_arrive(fb);
            }
            first = s - steps;
        }
        // copies in flight have to land before the CTA gives up its memory, also
        // where another warp gives up after this one's last copies
        for (uint32_t i = it > kStages ? it - kStages : mine; i < it; i += S::kSlotWarps)
            wait_drain(smem_u32(&full_bar[i % kStages]), (i / kStages) & 1);
    } else if (warp < kFirstEpiWarp) {
        // ---- scales to tensor memory: each warp to its lane quarter ----------------------
        // The tensor pipe's own copies (tcgen05.cp) run in line with the
        // products, about 100 cycles each and six a stage.
        const uint8_t *smem = dsmem + (smem_base - smem_u32(dsmem));
        const uint32_t sf0 = tmem + ((uint32_t)(warp & 3) << 21) + kSfCol;   // lane 32 (warp & 3)
        const int tiles = total > pair ? (total - pair - 1) / pairs + 1 : 0;
        const uint32_t done = PAIR ? cluster_map(smem_u32(&sf_bar[0]), 0) : smem_u32(&sf_bar[0]);
        bool ok = true;
        for (int it = 0; it < tiles * steps; ++it) {
            const uint32_t slot = it % kStages;
            ok = wait_bounded(smem_u32(&full_bar[slot]), (it / kStages) & 1, abort_flag,
                              args.status, MOE_DEV_TIMEOUT);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();   // the products that read these columns before are done
            const uint8_t *sc = smem + slot * kStageBytes + kSAOff + lane * 16;
            const uint32_t sf = sf0 + slot * kSfStage;
            // a K block: token rows, first and second weight block; what a
            // short stage leaves in place of one is not used
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                tmem_st4(sf + 12 * k, *reinterpret_cast<const uint4 *>(sc + k * 512));
                tmem_st4(sf + 12 * k + 4, *reinterpret_cast<const uint4 *>(sc + 1024 + k * 512));
                tmem_st4(sf + 12 * k + 8, *reinterpret_cast<const uint4 *>(sc + 2048 + k * 512));
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (elect_one()) {
                if constexpr (PAIR) mbar_arrive_cluster(done + slot * 8);
                else mbar_arrive(done + slot * 8);
            }
        }
    } else {
        // ---- epilogue ------------------------------------------------------------------
        // A warp has 32 rows (its lane quarter) and 32 features of SwiGLU, or 128
        // columns.  The accumulator is given back as soon as this warp's part
        // of it is in registers: the next tile's products run under the rest.
        const int q = warp & 3, part = (warp - kFirstEpiWarp) >> 2;
        const int m = 32 * q + lane;   // this thread's row of the tile
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16);
        const uint32_t given = PAIR ? cluster_map(smem_u32(&acc_empty), 0) : smem_u32(&acc_empty);
        uint32_t tiles = 0;
        for (int t = pair; t < total; t += pairs, ++tiles) {
            const Tile tl = decode<kTM>(t, rank, G, s_tiles, s_off);
            const bool ok = wait_bounded(smem_u32(&acc_full), tiles & 1, abort_flag, args.status,
                                         MOE_DEV_TIMEOUT);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const bool valid = m < tl.nvalid;
            const size_t row = (size_t)tl.row0 + m;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_cluster(given);
                    else mbar_arrive(given);
                }
            };
            if constexpr (SW) {
                uint32_t g[2][16], u[2][16];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    tmem_ld16(lane_base + part * 32 + p * 16, g[p]);
                    tmem_ld16(lane_base + 128 + part * 32 + p * 16, u[p]);
                }
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    tmem_wait_ld(g[p]);
                    tmem_wait_ld(u[p]);
                }
                release();
                float h[32];
                uint32_t amax = 0;
#pragma unroll
                for (int j = 0; j < 32; ++j) {   // a block of scales
                    h[j] = silu_mul(__uint_as_float(g[j / 16][j % 16]), __uint_as_float(u[j / 16][j % 16]));
                    amax = max(amax, __float_as_uint(h[j]) & 0x7fffffffu);
                }
                const uint32_t byte = mx4_scale_byte(amax);
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = h[8 * j + i];
                    o[j] = mx4_codes8(v, byte);
                }
                if (valid) {
                    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(args.c) + row * (args.n_out / 4) +
                                               tl.nt * 64 + part * 16) = make_uint4(o[0], o[1], o[2], o[3]);
                    args.h_scales[row * (args.n_out / 64) + tl.nt * 4 + part] = (uint8_t)byte;
                }
            } else if (2 * tl.nt + part >= nblocks) {
                release();   // no second weight block
            } else if (args.c_bf16) {
                uint32_t w[64];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    uint32_t r[2][16];
                    tmem_ld16(lane_base + part * 128 + p * 32, r[0]);
                    tmem_ld16(lane_base + part * 128 + p * 32 + 16, r[1]);
                    tmem_wait_ld(r[0]);
                    tmem_wait_ld(r[1]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[i / 8][2 * i % 16]),
                                                                 __uint_as_float(r[i / 8][2 * i % 16 + 1]));
                        w[16 * p + i] = *reinterpret_cast<uint32_t *>(&b);
                    }
                }
                release();
                uint16_t *o = static_cast<uint16_t *>(args.c) + row * args.n_out + tl.nt * kTN + part * 128;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint32_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = w[8 * j + i];
                    if (valid) store32(o + 16 * j, v);
                }
            } else {
                float *o = static_cast<float *>(args.c) + row * args.n_out + tl.nt * kTN + part * 128;
#pragma unroll
                for (int q4 = 0; q4 < 2; ++q4) {   // 64 columns at a time
                    uint32_t r[4][16];
#pragma unroll
                    for (int j = 0; j < 4; ++j) tmem_ld16(lane_base + part * 128 + q4 * 64 + j * 16, r[j]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) tmem_wait_ld(r[j]);
                    if (q4 == 1) release();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = r[j >> 1][8 * (j & 1) + i];
                        if (valid) store32(o + q4 * 64 + 8 * j, v);
                    }
                }
            }
        }
    }

    // neither CTA of a pair leaves while the other's products read its memory
    // or its arrivals are on their way
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
    if (warp == kMmaWarp) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc2(tmem, kTmemCols);
        else tmem_dealloc(tmem, kTmemCols);
    }
}

template <bool SW, bool PAIR>
int launch(const Mx4Args &args, const void *a, cudaStream_t s) {
    using S = Shape<SW, PAIR>;
    auto kern = mx4_gemm_kernel<SW, PAIR>;
    cudaLaunchConfig_t c = {};
    c.blockDim = dim3(S::kThreads);
    c.dynamicSmemBytes = S::kSmemBytes;
    c.stream = s;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = PAIR ? 2 : 1;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;

    static std::once_flag once[64];
    static int rc[64], clusters[64];   // as many as run at the same time
    int dev = 0;
    MOE_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return cuda_fail("device ordinal beyond 63");
    std::call_once(once[dev], [&] {
        rc[dev] = (int)cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes);
        clusters[dev] = sm_count();
        if (!PAIR || rc[dev]) return;
        cudaLaunchConfig_t q = c;
        q.gridDim = dim3((unsigned)(sm_count() / 2 * 2));
        q.numAttrs = 1;
        rc[dev] = (int)cudaOccupancyMaxActiveClusters(&clusters[dev], kern, &q);
        if (!rc[dev] && clusters[dev] < 1) rc[dev] = (int)cudaErrorInvalidConfiguration;
    });
    if (rc[dev]) return cuda_fail("setting up the MXFP4 product", (cudaError_t)rc[dev]);
    CUtensorMap tmA, tmA32;
    if (!encode_2d(&tmA, a, true, (uint64_t)args.k_dim / 2, (uint64_t)args.rows, 64) ||
        !encode_2d(&tmA32, a, true, (uint64_t)args.k_dim / 2, (uint64_t)args.rows, 32))
        return cuda_fail("cuTensorMapEncodeTiled (activations)");
    const int64_t nt = ceil_div(args.n_out, kTN);
    const int64_t bound = nt * (args.groups + ceil_div(args.rows, S::kTM));
    c.gridDim = dim3((PAIR ? 2 : 1) * (unsigned)std::min<int64_t>(clusters[dev], bound));
    c.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&c, kern, tmA, tmA32, args);
    return e == cudaSuccess ? MOE_OK : cuda_fail("cudaLaunchKernelEx", e);
}

// Pairs where a group has more than one CTA's 128 rows on average: the second
// CTA's products are wasted on a smaller one.  (CTAs alone / pairs: 273 rows in
// 33 groups 42 / 52 us, 264 with SwiGLU 82 / 88; 4599 in 33 with SwiGLU 98 / 99;
// 16411 in 8 groups 124 / 113, 8192 with SwiGLU in 4 95 / 84.)
template <bool SW>
int launch(const Mx4Args &args, const void *a, cudaStream_t s) {
    return args.rows > (int64_t)128 * args.groups ? launch<SW, true>(args, a, s) : launch<SW, false>(args, a, s);
}

}  // namespace

int launch_mx4_gemm(int groups, int n_out, int k_dim, int rows, const void *a, const void *a_scales,
                    const int32_t *offsets, const void *w, const void *w_scales, void *c, int c_dtype,
                    int32_t *status, cudaStream_t s) {
    Mx4Args args = {};
    args.groups = groups;
    args.n_out = n_out;
    args.k_dim = k_dim;
    args.rows = rows;
    args.a_scales = static_cast<const uint8_t *>(a_scales);
    args.offsets = offsets;
    args.w = static_cast<const uint8_t *>(w);
    args.w_scales = static_cast<const uint8_t *>(w_scales);
    args.c = c;
    args.c_bf16 = c_dtype == MOE_OUT_BF16;
    args.status = status;
    return launch<false>(args, a, s);
}

int launch_mx4_gemm_swiglu(int groups, int inter, int k_dim, int rows, const void *a,
                           const void *a_scales, const int32_t *offsets, const void *w13,
                           const void *w13_scales, void *h, void *h_scales, int32_t *status,
                           cudaStream_t s) {
    Mx4Args args = {};
    args.groups = groups;
    args.n_out = 2 * inter;
    args.k_dim = k_dim;
    args.rows = rows;
    args.a_scales = static_cast<const uint8_t *>(a_scales);
    args.offsets = offsets;
    args.w = static_cast<const uint8_t *>(w13);
    args.w_scales = static_cast<const uint8_t *>(w13_scales);
    args.c = h;
    args.h_scales = static_cast<uint8_t *>(h_scales);
    args.status = status;
    return launch<true>(args, a, s);
}

}  // namespace moe
