// The paged cache around attention: the tables of a step, and the values that
// slots of the cache hold.
//
// cache_tables: with new[b] tokens for a request that holds held[b],
//   need[b]  = ceil((held + new) / page) - ceil(held / page)
//   starts   = exclusive sum of new,   first[b] = exclusive sum of need
//   page i of a request's new ones = free[(next + first[b] + i) mod F]
//   token t of request b (the largest with starts[b] <= t) stands at
//   position held[b] + t - starts[b].
// Bound by latency: a step's tables are some kilobytes.  Each CTA of one
// cluster sums all of the requests itself (no sums to pass on) and writes its
// share of the tokens and pages, after a barrier of the cluster: by then every
// CTA has read what outputs may replace (held, the free range).  Eight requests
// take 4.6 us in a graph (8.3 where each call is the host's), 1000 that decode or have up to 96
// new tokens 6.4.
// One CTA up to 4096 token rows, eight above.
//
// cache_read: a thread to 16 bytes of output; bound by memory, 3 us for the 5001 rows of 4 heads of
// 64 that a prompt writes.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "mx4.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kTabThreads = 1024, kTabMaxRequests = 16384;

struct TabArgs {
    int B, page_shift, free_count, max_pages, max_tokens;
    const int32_t *held, *fresh, *free_pages;
    const int64_t *free_range;
    int32_t *table, *lengths, *starts, *slots, *positions;
    int64_t *free_out;
    int32_t *status;
};

// Inclusive sums over the CTA of two numbers a thread; sh holds 2 x 32.
__device__ __forceinline__ void block_scan2(int64_t &a, int64_t &b, int64_t (*sh)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) a += x, b += y;
    }
    __syncthreads();   // the words of an earlier call have been read
    if (lane == 31) sh[0][warp] = a, sh[1][warp] = b;
    __syncthreads();
    int64_t x = sh[0][lane], y = sh[1][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t p = __shfl_up_sync(0xffffffffu, x, o), q = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) x += p, y += q;
    }
    const int before = max(warp - 1, 0);
    const int64_t pa = __shfl_sync(0xffffffffu, x, before), pb = __shfl_sync(0xffffffffu, y, before);
    if (warp > 0) a += pa, b += pb;
}

// The largest b < n with v[b] <= t (v does not decrease, v[0] = 0).
__device__ __forceinline__ int last_at_most(const int *v, int n, int t) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Whether page `id`'s slots are numbers.
__device__ __forceinline__ bool is_page(int id, int page_shift) { return (unsigned)id <= (unsigned)(INT32_MAX >> page_shift); }

// One cluster.  Shared memory: starts [B + 1], first [B + 1], held [B].
__global__ void __launch_bounds__(kTabThreads) cache_tables_kernel(const TabArgs a) {
    extern __shared__ int s_tab[];
    __shared__ int64_t sh[2][32];
    __shared__ int64_t s_sum[2];
    int *s_start = s_tab, *s_first = s_tab + a.B + 1, *s_held = s_first + a.B + 1;
    const int tid = threadIdx.x, rank = blockIdx.x, ranks = gridDim.x;
    const int page = 1 << a.page_shift;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int64_t next = a.free_range[0], end = a.free_range[1];
    bool bad = false, full = false;
    int64_t tokens = 0, pages = 0;   // of the requests before these
    for (int b0 = 0; b0 < a.B; b0 += kTabThreads) {
        const int b = b0 + tid;
        int held = 0, fresh = 0, had = 0, want = 0;
        if (b < a.B) {
            held = a.held[b];
            fresh = a.fresh[b];
            const int64_t total = (int64_t)held + fresh;
            if (held < 0 || fresh < 0 || total > INT32_MAX - 256) bad = true, held = fresh = 0;
            had = (held + page - 1) >> a.page_shift;
            want = (held + fresh + page - 1) >> a.page_shift;
            if (want > a.max_pages) full = true;
            // tokens that join the last held page take its id from the table
            else if (fresh > 0 && (held & (page - 1)) && !is_page(a.table[(int64_t)b * a.max_pages + had - 1], a.page_shift))
                bad = true;
        }
        int64_t t = fresh, p = want - had;
        block_scan2(t, p, sh);
        if (b < a.B) {
            // values beyond 32 bits are those of a step that is not made
            s_start[b] = (int)(tokens + t - fresh);
            s_first[b] = (int)(pages + p - (want - had));
            s_held[b] = held;
        }
        if (tid == kTabThreads - 1) s_sum[0] = t, s_sum[1] = p;
        __syncthreads();
        tokens += s_sum[0];
        pages += s_sum[1];
        // the next round's writes of s_sum come behind block_scan2's barriers
    }
    if (tokens > a.max_tokens || pages > end - next || next < 0 || end - next > a.free_count) full = true;
    const bool any_bad = __syncthreads_or(bad), any_full = __syncthreads_or(full);
    const bool fail = any_bad || any_full;
    if (fail) tokens = pages = 0;
    if (tid == 0) s_start[a.B] = (int)tokens, s_first[a.B] = (int)pages;
    __syncthreads();
    ptx::cluster_sync();
    if (rank == 0 && tid == 0) {
        if (a.status && fail) atomicOr(a.status, (any_bad ? MOE_DEV_BAD_INDEX : 0) | (any_full ? MOE_DEV_NO_ROOM : 0));
        a.free_out[0] = next + pages;
        a.free_out[1] = end;
    }
    const int step = ranks * kTabThreads, first = rank * kTabThreads + tid;
    for (int b = first; b <= a.B; b += step) {
        a.starts[b] = fail ? 0 : s_start[b];
        // after a failed step the value read is not s_held's where it was bad
        if (b < a.B && !(fail && a.lengths == a.held))
            a.lengths[b] = fail ? a.held[b] : s_held[b] + s_start[b + 1] - s_start[b];
    }
    const unsigned F = (unsigned)max(a.free_count, 1), at = (unsigned)((uint64_t)next % F);
    for (int f = first; f < (int)pages; f += step) {
        const int b = last_at_most(s_first, a.B + 1, f);
        const int had = (s_held[b] + page - 1) >> a.page_shift;
        a.table[(int64_t)b * a.max_pages + had + f - s_first[b]] = a.free_pages[((uint64_t)at + f) % F];
    }
    for (int t = first; t < a.max_tokens; t += step) {
        int slot = -1, pos = 0;
        if (t < (int)tokens) {
            const int b = last_at_most(s_start, a.B + 1, t);
            pos = s_held[b] + t - s_start[b];
            const int i = pos >> a.page_shift, had = (s_held[b] + page - 1) >> a.page_shift;
            const int id = i < had ? a.table[(int64_t)b * a.max_pages + i]
                                   : a.free_pages[((uint64_t)at + s_first[b] + i - had) % F];
            slot = is_page(id, a.page_shift) ? (id << a.page_shift) + (pos & (page - 1)) : INT32_MIN;
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
}

// One 16-byte piece of the output (eight values) a thread.
__global__ void __launch_bounds__(256)
    cache_read_kernel(const uint32_t *codes, const uint8_t *scales, int page_shift, int heads, int n8,
                      int64_t slots_in_cache, int64_t total, const int32_t *slots, uint4 *k, uint4 *v,
                      int32_t *status) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    const int per_row = heads * n8;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t row = i / per_row;
        const int rest = (int)(i - row * per_row), h = rest / n8, c = rest - h * n8;
        const int slot = slots[row];
        if (slot < 0 || slot >= slots_in_cache) {
            if (slot != -1 && status && rest == 0) atomicOr(status, MOE_DEV_BAD_INDEX);
            continue;
        }
        const int64_t p = slot >> page_shift;
        const int64_t at = ((p * 2 * heads + h) << page_shift) + (slot & ((1 << page_shift) - 1));
        const int64_t kv = (int64_t)heads << page_shift;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint4 *out = j ? v : k;
            if (!out) continue;
            const int64_t r = at + j * kv;
            const uint32_t code = codes[r * n8 + c];
            const float sc = mx4_scale(scales[(r * n8 + c) >> 2]);
            float f[8];
            mx4_values8(code, sc, f);
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * q], f[2 * q + 1]);
                w[q] = *reinterpret_cast<const uint32_t *>(&b);
            }
            out[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

int shift_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

}  // namespace

int launch_cache_tables(int B, int page, const int32_t *held, const int32_t *fresh,
                        const int32_t *free_pages, int free_count, const int64_t *free_range,
                        int32_t *table, int max_pages, int32_t *lengths, int32_t *starts,
                        int32_t *slots, int32_t *positions, int max_tokens, int64_t *free_out,
                        int32_t *status, cudaStream_t s) {
    TabArgs a;
    a.B = B;
    a.page_shift = shift_of(page);
    a.free_count = free_count;
    a.max_pages = max_pages;
    a.max_tokens = max_tokens;
    a.held = held;
    a.fresh = fresh;
    a.free_pages = free_pages;
    a.free_range = free_range;
    a.table = table;
    a.lengths = lengths;
    a.starts = starts;
    a.slots = slots;
    a.positions = positions;
    a.free_out = free_out;
    a.status = status;
    const size_t smem = sizeof(int) * (3 * (size_t)B + 2);
    if (smem > 40 * 1024)   // the most that any call takes: calls of several threads set the same
        MOE_CUDA_TRY(cudaFuncSetAttribute(cache_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)sizeof(int) * (3 * kTabMaxRequests + 2)));
    cudaLaunchConfig_t c = {};
    const unsigned ctas = max_tokens > 4 * kTabThreads ? 8 : 1;
    c.gridDim = dim3(ctas);
    c.blockDim = dim3(kTabThreads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&c, cache_tables_kernel, (const TabArgs)a);
    return e == cudaSuccess ? MOE_OK : cuda_fail("cudaLaunchKernelEx", e);
}

int launch_cache_read(const moe_cache4 *cache, int n, const int32_t *slots, void *k, void *v,
                      int32_t *status, cudaStream_t s) {
    const int n8 = cache->dim / 8;
    const int64_t total = (int64_t)n * cache->kv_heads * n8;
    const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(total, 256), (int64_t)sm_count() * 16);
    return launch_dependent(cache_read_kernel, dim3(grid), dim3(256), 0, s,
                            static_cast<const uint32_t *>(cache->codes),
                            static_cast<const uint8_t *>(cache->scales), shift_of(cache->page),
                            (int)cache->kv_heads, n8, (int64_t)cache->pages * cache->page, total, slots,
                            static_cast<uint4 *>(k), static_cast<uint4 *>(v), status);
}

}  // namespace moe
