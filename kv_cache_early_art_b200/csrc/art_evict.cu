// art_evict.cu -- eviction from the paged cache by accumulated attention
// weight (art_cache_evict in art.h).
//
// Of the L cached tokens of a (sequence, kv-head) unit, n = min(L, budget)
// stay: the first `sink`, the last `recent`, and of the others those with the
// largest accumulated weight, equal weights oldest first.  They keep their
// order (a walk from the newest to the oldest page still means that), so
// token kept[i] moves to row i, kept[i] >= i.
//
// Two kernels.  art_evict_select_kernel, a cluster of up to 8 CTAs a unit: the
// weights are read once into the cluster's shared memory as order-preserving
// keys; three radix steps (11, 11 and 10 bits), their histograms summed
// through distributed shared memory, give the smallest kept key exactly; a
// prefix sum over the kept flags gives every kept token its row.  No sort, no atomics
// that decide an order: the result is exact and reproducible.
// Then the kept rows of K and V move (few of them still in the selection
// kernel), bound by HBM: each read once and written once.  To new pages (art_evict_move_kernel) all rows move
// independently.  In place (art_evict_slide_kernel) the rows of a unit move
// front to back: a cluster owns a column slice of one unit's K or V, reads a
// run of rows into registers and, behind a barrier, writes it; since kept[i]
// >= i, no write reaches a row that a later run still has to read, so nothing
// but that barrier orders it.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/art.h"
#include "art_host.h"
#include "art_stream.cuh"

namespace {

namespace cg = cooperative_groups;
using art_host::aligned;
using art_host::apart;
using art_host::elem_size;
using art_host::is_null;

constexpr int kSelThreads = 512;     // two CTAs an SM: with 1024 threads the last clusters of 8 had to wait
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kSliceTokens = 49152;     // weights a CTA holds (192 KB)
constexpr int kBins = 2048;
constexpr int kSelBatch = 4;             // keys
constexpr int kMoveThreads = 256;
constexpr int kRunRows = 64;            // rows a CTA moves to new pages
constexpr int kWholeRows = 512;         // most rows the selection kernel moves itself
static_assert(kWholeRows <= kSelThreads && kWholeRows * 16 <= 3 * 2048 * 4, "a thread and a place a row");
constexpr int kSlideRows = 128;         // rows a CTA holds at a time in place
constexpr int kSlideVecs = 8;           // 16-byte columns of its slice, at most

struct EvictArgs {
    uint8_t *k, *v;
    int64_t ks0, ks1, ks2, vs0, vs1, vs2;   // page, head, token strides (bytes)
    const int32_t *pt, *npt;                // npt == pt: in place
    int64_t pts0, npts0;
    const int32_t *sl;
    const float *mass;
    int64_t ms0, ms1;
    float *nmass;
    int64_t ns0, ns1;
    int64_t nwidth;                         // columns of nmass
    int32_t *nsl, *kept;
    int64_t kp0, kp1;
    int Hkv, page, max_blocks, num_pages, budget, sink, recent;
    int cluster;
    int in_place, whole;        // whole: the selection kernel moves the rows too
    int row_vecs, lanes;        // 16-byte pieces of a row; threads on one row
    int slices, slide_cluster;  // in place: column slices of a row, CTAs on each
    int64_t runs;               // to new pages: runs of kRunRows rows
    int32_t *status;
};

__device__ __forceinline__ void report(int32_t *status, int32_t code)
{
    if (status)
        atomicCAS(status, 0, code);
}

__device__ __forceinline__ int length_of(const EvictArgs &a, int b)
{
    const int64_t cap = (int64_t)a.max_blocks * a.page;
    const int L = a.sl[b];
    return L <= 0 ? 0 : (int)(L < cap ? L : cap);
}

// Larger weight, larger key; -0 joins +0 and a NaN ranks below everything.
__device__ __forceinline__ uint32_t key_of(float w)
{
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
    return w != w ? 0u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float weight_of(uint32_t k)
{
    return __uint_as_float(k == 0u ? 0x7fc00000u : k ^ (~(uint32_t)((int32_t)k >> 31) | 0x80000000u));
}

// Where a kept row comes from and goes to: pages and rows within them; a
// negative page: it stays, or cannot be moved.
struct Move {
    int sp, so, dp, dof;
};

__device__ __forceinline__ Move move_of(const EvictArgs &a, int b, const int32_t *krow, int i, bool tell)
{
    Move m = {-1, 0, -1, 0};
    const int src = krow[i];
    if (a.in_place && src == i)
        return m;
    const int sb = src / a.page, db = i / a.page;
    const int32_t *from = a.pt + (int64_t)b * a.pts0;
    const int sp = from[sb], dp = a.npt[(int64_t)b * a.npts0 + db];
    // (i <= src: block db is one of the sequence's; its own page is no new page)
    const bool own = !a.in_place && dp == from[db];
    if (sp < 0 || sp >= a.num_pages || dp < 0 || dp >= a.num_pages || own) {
        if (tell)
            report(a.status, ART_ERR_BAD_INDEX);
        return m;
    }
    return {sp, src - sb * a.page, dp, i - db * a.page};
}

// A CTA of THREADS threads moves `rows` kept rows of a unit, K and V, from the
// lo-th on, to new pages; at: a place in shared memory for each.
template <int THREADS>
__device__ __forceinline__ void move_rows(const EvictArgs &a, int b, int h, int lo, int rows, Move *at)
{
    if (threadIdx.x < rows)
        at[threadIdx.x] = move_of(a, b, a.kept + (int64_t)b * a.kp0 + (int64_t)h * a.kp1, lo + threadIdx.x, h == 0);
    __syncthreads();
    const int lane = threadIdx.x % a.lanes, r0 = threadIdx.x / a.lanes, step = THREADS / a.lanes;
    uint8_t *kb = a.k + (int64_t)h * a.ks1, *vb = a.v + (int64_t)h * a.vs1;
    for (int c = lane; c < a.row_vecs; c += a.lanes) {
#pragma unroll 4
        for (int r = r0; r < rows; r += step) {
            const Move m = at[r];
            if (m.sp >= 0) {
                const uint4 x = *reinterpret_cast<const uint4 *>(kb + m.sp * a.ks0 + m.so * a.ks2 + c * 16);
                const uint4 y = *reinterpret_cast<const uint4 *>(vb + m.sp * a.vs0 + m.so * a.vs2 + c * 16);
                *reinterpret_cast<uint4 *>(kb + m.dp * a.ks0 + m.dof * a.ks2 + c * 16) = x;
                *reinterpret_cast<uint4 *>(vb + m.dp * a.vs0 + m.dof * a.vs2 + c * 16) = y;
            }
        }
    }
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads, 2) art_evict_select_kernel(const __grid_constant__ EvictArgs a)
{
    extern __shared__ __align__(16) uint32_t keys[];                 // this CTA's slice of the tokens
    __shared__ __align__(16) uint32_t hist[3][kBins];   // counts by digit, a step each
    __shared__ uint2 packed[2][kBins / 4];             // a step's counts for the cluster, 16 bits each
    __shared__ uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
    __shared__ __align__(8) uint32_t cta_sum[2];
    __shared__ uint32_t found[2];                      // digit, tokens still wanted among its ties
    art_stream::follow();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = CLUSTER ? a.cluster : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
    const int unit = blockIdx.x / C, b = unit / a.Hkv, h = unit - b * a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = length_of(a, b);
    for (int i = tid; i < 3 * kBins / 4; i += kSelThreads)
        reinterpret_cast<uint4 *>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    const int n = L < a.budget ? L : a.budget;
    const float *mrow = a.mass + (int64_t)b * a.ms0 + (int64_t)h * a.ms1;
    float *nrow = a.nmass + (int64_t)b * a.ns0 + (int64_t)h * a.ns1;
    int32_t *krow = a.kept + (int64_t)b * a.kp0 + (int64_t)h * a.kp1;
    const int per = ((L + C - 1) / C + 31) / 32 * 32;
    const int first = min(L, rank * per), count = min(L, first + per) - first;
    if (rank == 0 && h == 0 && tid == 0) {
        a.nsl[b] = n;
        if (a.sl[b] > L)
            report(a.status, ART_ERR_BAD_INDEX);
    }
    // a warp keeps to its segment of the slice
    const int seg = ((count + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int s0 = min(count, warp * seg), s1 = min(count, s0 + seg);
    // the tokens the weights decide about: [lo, hi) of the slice; all others stay
    const bool every = n == L;                         // the same for the whole cluster, as is `want`
    const int lo = every ? count : max(0, min(count, a.sink - first));
    const int hi = every ? count : max(lo, min(count, L - a.recent - first));
    uint32_t want = every ? 0u : (uint32_t)(n - a.sink - a.recent), edge = 0xffffffffu;
    const bool search = want > 0;
    // of them in the warp's segment (the bounds tested key by key: 2 us of those 75)
    const int d0 = min(max(s0, lo), s1), d1 = max(d0, min(s1, hi));
    // the whole segment is requested before any of it is looked at (16 units of up to
    // 131072 to 16384: 74.5 us with 4 bytes a request, 73.2 with 16)
    int i4 = s0;
    if (reinterpret_cast<uintptr_t>(mrow) % 16 == 0) {   // (a segment starts at a multiple of 32)
        i4 = max(s0, s1 / 4 * 4);
        for (int i = s0 + 4 * lane; i < i4; i += 128)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(keys + i)),
                         "l"(mrow + first + i)
                         : "memory");
    }
    for (int i = i4 + lane; i < s1; i += 32)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(keys + i)),
                     "l"(mrow + first + i)
                     : "memory");
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    __syncthreads();                                   // hist is clear, every copy in
    for (int i0 = s0 + lane; i0 < s1; i0 += 32 * kSelBatch) {
#pragma unroll
        for (int j = 0; j < kSelBatch; ++j) {
            const int i = i0 + 32 * j;
            if (i < s1) {
                const uint32_t k = key_of(__uint_as_float(keys[i]));
                keys[i] = k;
                if (search && i >= lo && i < hi)
                    atomicAdd(&hist[0][k >> 21], 1u);
            }
        }
    }
    if (search) {
        edge = 0u;
#pragma unroll
        for (int step = 0; step < 3; ++step) {
            // digits: bits 31-21, 20-10, 9-0
            if (step > 0) {
                const int above = step == 1 ? 21 : 10, shift = step == 1 ? 10 : 0;
                const uint32_t bits = step == 1 ? 2047u : 1023u, prefix = edge << above;
                for (int i0 = d0 + lane; i0 < d1; i0 += 32 * kSelBatch) {
                    uint32_t k[kSelBatch];
#pragma unroll
                    for (int j = 0; j < kSelBatch; ++j)
                        k[j] = i0 + 32 * j < d1 ? keys[i0 + 32 * j] : ~prefix;
#pragma unroll
                    for (int j = 0; j < kSelBatch; ++j)
                        if (((k[j] ^ prefix) >> above) == 0u)
                            atomicAdd(&hist[step][(k[j] >> shift) & bits], 1u);
                }
            }
            __syncthreads();
            // thread t holds bins 2047 - 4 t down to 2044 - 4 t of the whole unit
            const int quad = kBins / 4 - 1 - tid;
            uint4 c = reinterpret_cast<const uint4 *>(hist[step])[quad];
            if (CLUSTER) {
                packed[step & 1][quad] = make_uint2(c.x | (c.y << 16), c.z | (c.w << 16));
                cluster.sync();
                uint2 x[kMaxCluster - 1];              // the other CTAs', all in flight at once
#pragma unroll
                for (int j = 0; j < kMaxCluster - 1; ++j) {
                    x[j] = make_uint2(0u, 0u);
                    if (j + 1 < C)
                        x[j] = cluster.map_shared_rank(packed[step & 1], rank + j + 1 < C ? rank + j + 1 : rank + j + 1 - C)[quad];
                }
#pragma unroll
                for (int j = 0; j < kMaxCluster - 1; ++j) {
                    c.x += x[j].x & 0xffffu;
                    c.y += x[j].x >> 16;
                    c.z += x[j].y & 0xffffu;
                    c.w += x[j].y >> 16;
                }
            }
            const uint32_t mine = c.x + c.y + c.z + c.w;
            uint32_t inc = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o)
                    inc += y;
            }
            if (lane == 31)
                warp_gt[warp] = inc;
            __syncthreads();
            const uint32_t others = __reduce_add_sync(0xffffffffu, lane < warp ? warp_gt[lane & (kSelWarps - 1)] : 0u);
            const uint32_t upto = others + inc;
            if (upto >= want && upto - mine < want) {
                uint32_t above = upto - mine;
                int d = kBins - 1 - 4 * tid;
                const uint32_t n4[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (d == kBins - 1 - 4 * tid - j && above + n4[j] < want) {
                        above += n4[j];
                        --d;
                    }
                found[0] = (uint32_t)d;
                found[1] = want - above;
            }
            __syncthreads();
            edge = (edge << (step == 2 ? 10 : 11)) | found[0];
            want = found[1];
        }
    }
    // edge: the smallest key that stays; of its ties the `want` oldest do
    uint32_t gt = 0, eq = 0;
    __syncwarp();
    for (int i0 = d0 + lane; i0 < d1; i0 += 32 * kSelBatch) {
        uint32_t k[kSelBatch];
#pragma unroll
        for (int j = 0; j < kSelBatch; ++j)
            k[j] = i0 + 32 * j < d1 ? keys[i0 + 32 * j] : 0u;
#pragma unroll
        for (int j = 0; j < kSelBatch; ++j) {
            gt += k[j] > edge ? 1u : 0u;
            eq += k[j] == edge && i0 + 32 * j < d1 ? 1u : 0u;
        }
    }
    if (lane == 0)
        gt += (uint32_t)(s1 - s0 - (d1 - d0));           // those that stay whatever they weigh
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        warp_gt[warp] = gt;
        warp_eq[warp] = eq;
    }
    __syncthreads();
    const uint32_t wg = lane < kSelWarps ? warp_gt[lane] : 0u, we = lane < kSelWarps ? warp_eq[lane] : 0u;
    // larger keys and ties before this warp's segment
    uint32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? wg : 0u);
    uint32_t eb = __reduce_add_sync(0xffffffffu, lane < warp ? we : 0u);
    if (CLUSTER) {
        if (warp == 0) {
            const uint32_t sg = __reduce_add_sync(0xffffffffu, wg), se = __reduce_add_sync(0xffffffffu, we);
            if (lane == 0) {
                cta_sum[0] = sg;
                cta_sum[1] = se;
            }
        }
        cluster.sync();
        uint32_t og = 0, oe = 0;                       // the lower ranks' sums, a lane each
        if (lane < rank) {
            const uint2 o = *reinterpret_cast<const uint2 *>(cluster.map_shared_rank(&cta_sum[0], lane));
            og = o.x;
            oe = o.y;
        }
        at += __reduce_add_sync(0xffffffffu, og);
        eb += __reduce_add_sync(0xffffffffu, oe);
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");   // waited for before leaving
    }
    at += min(eb, want);
    const uint32_t below = (1u << lane) - 1u;
    // (a batch's keys are read before any store, which could alias them)
    for (int i0 = s0; i0 < s1; i0 += 32 * kSelBatch) {
        uint32_t k[kSelBatch];
        unsigned stay[kSelBatch], ties[kSelBatch];
#pragma unroll
        for (int j = 0; j < kSelBatch; ++j) {
            const int i = i0 + 32 * j + lane;
            k[j] = i < s1 ? keys[i] : 0u;
            const bool in = i < s1, safe = i < lo || i >= hi;
            stay[j] = __ballot_sync(0xffffffffu, in && (safe || k[j] > edge));
            ties[j] = __ballot_sync(0xffffffffu, in && !safe && k[j] == edge);
        }
#pragma unroll
        for (int j = 0; j < kSelBatch; ++j) {
            if (ties[j]) {                             // the same for the warp
                const bool tie = (ties[j] >> lane) & 1;
                stay[j] |= __ballot_sync(0xffffffffu, tie && eb + __popc(ties[j] & below) < want);
                eb += __popc(ties[j]);
            }
            if ((stay[j] >> lane) & 1) {
                const uint32_t pos = at + __popc(stay[j] & below);
                krow[pos] = first + i0 + 32 * j + lane;
                nrow[pos] = weight_of(k[j]);
            }
            at += __popc(stay[j]);
        }
    }
    for (int64_t i = n + rank * kSelThreads + tid; i < a.nwidth; i += C * kSelThreads)
        nrow[i] = 0.f;
    for (int i = n + rank * kSelThreads + tid; i < a.budget; i += C * kSelThreads)
        krow[i] = -1;
    if (CLUSTER)                                       // nobody leaves while its sums are read
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (!CLUSTER && a.whole) {
        // few rows to new pages: moved here, their places over the counts
        __syncthreads();
        move_rows<kSelThreads>(a, b, h, 0, n, reinterpret_cast<Move *>(hist));
    }
}

// To new pages: a CTA moves kRunRows rows of one unit, K and V.
__global__ void __launch_bounds__(kMoveThreads) art_evict_move_kernel(const __grid_constant__ EvictArgs a)
{
    __shared__ Move at[kRunRows];
    art_stream::follow();
    const int unit = (int)(blockIdx.x / a.runs), b = unit / a.Hkv, h = unit - b * a.Hkv;
    const int n = a.nsl[b];
    const int lo = (int)(blockIdx.x % a.runs) * kRunRows, rows = min(kRunRows, n - lo);
    if (rows <= 0)
        return;
    move_rows<kMoveThreads>(a, b, h, lo, rows, at);
}

// In place: the CTAs of a cluster slide one column slice of one unit's K or V
// to the front, a run of rows each at a time.
__global__ void __launch_bounds__(kMoveThreads) art_evict_slide_kernel(const __grid_constant__ EvictArgs a)
{
    constexpr int kMost = kSlideRows * kSlideVecs / kMoveThreads;
    // the places of a run, of the one before (still being written by the slower
    // threads) and of the one after
    __shared__ Move places[3][kSlideRows];
    art_stream::follow();
    const int C = a.slide_cluster;
    int64_t x = blockIdx.x / C;
    const int rank = (int)(blockIdx.x - x * C);
    const int slice = (int)(x % a.slices);
    x /= a.slices;
    const bool values = x & 1;
    const int unit = (int)(x >> 1), b = unit / a.Hkv, h = unit - b * a.Hkv;
    const int n = a.nsl[b];
    const int64_t s0 = values ? a.vs0 : a.ks0, s2 = values ? a.vs2 : a.ks2;
    const int lane = threadIdx.x % a.lanes, r0 = threadIdx.x / a.lanes, step = kMoveThreads / a.lanes;
    uint8_t *base = (values ? a.v + (int64_t)h * a.vs1 : a.k + (int64_t)h * a.ks1) + ((int64_t)slice * a.lanes + lane) * 16;
    const int32_t *krow = a.kept + (int64_t)b * a.kp0 + (int64_t)h * a.kp1;
    const bool tell = slice == 0 && !values && h == 0;
    const int rows = step * kMost < kSlideRows ? step * kMost : kSlideRows;   // a CTA's run
    auto look = [&](Move *at, int lo) {
        if (threadIdx.x < rows && lo + threadIdx.x < n)
            at[threadIdx.x] = move_of(a, b, krow, lo + threadIdx.x, tell);
    };
    look(places[0], rank * rows);
    __syncthreads();
    int now = 0;
    for (int all = 0; all < n; all += rows * C) {        // the same for the whole cluster
        const int lo = all + rank * rows, next = now == 2 ? 0 : now + 1;
        const Move *at = places[now];
        uint4 d[kMost];
#pragma unroll
        for (int j = 0; j < kMost; ++j) {
            const int r = r0 + j * step;
            if (r < rows && lo + r < n && at[r].sp >= 0)
                d[j] = *reinterpret_cast<const uint4 *>(base + at[r].sp * s0 + at[r].so * s2);
        }
        look(places[next], lo + rows * C);
        // the cluster's runs are in registers: they may be written
        if (C > 1)
            asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
        else
            __syncthreads();
#pragma unroll
        for (int j = 0; j < kMost; ++j) {
            const int r = r0 + j * step;
            if (r < rows && lo + r < n && at[r].sp >= 0)
                *reinterpret_cast<uint4 *>(base + at[r].dp * s0 + at[r].dof * s2) = d[j];
        }
        now = next;
    }
}

// --------------------------------------------------------------- host ----

// How many clusters of C selection CTAs the current device holds with an SM for
// each CTA: a cluster keeps to one group of SMs, so fewer than SMs / C (on a
// B200 33 of four, 22 of six, 15 of eight).
int clusters_at_once(int C)
{
    static std::atomic<int> known[16][kMaxCluster + 1];        // 1 + the answer; 0: not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 0;
    const bool keep = dev >= 0 && dev < 16;
    if (keep && known[dev][C].load(std::memory_order_relaxed) > 0)
        return known[dev][C].load(std::memory_order_relaxed) - 1;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)C);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = kSliceTokens * 4;                   // no two on an SM
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(art_evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSliceTokens * 4) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, art_evict_select_kernel<true>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (keep)
        known[dev][C].store(n + 1, std::memory_order_relaxed);
    return n;
}

bool has(const art_tensor_t &t) { return t.data != nullptr; }

// The CTAs of a unit of S tokens: what takes least time, a CTA for its slice and,
// where there are several, for the exchanges between them (about 5 us, as much as
// 8192 tokens), times the rounds in which all units find SMs to themselves
// (sharing them takes as long); no more than 4096-token slices ask for.  Measured,
// 64 tokens kept: 16 units of 16384 13.0 us in four slices, 14.5 in one, 14.1 in
// six; 16 of 131072 24.7 in six, 29.4 in eight; 40 of 65536 23.5 in three, 29.0
// in two or four; 64 of 131072 56 in four, 68 in three; 256 of 8192 16.9 in one,
// 29.5 in two.
int slices_of(int64_t S, int64_t units)
{
    int best = kMaxCluster;
    int64_t least = INT64_MAX;
    for (int C = 1; C <= kMaxCluster; ++C) {
        const int64_t slice = (S + C - 1) / C;
        if (slice > kSliceTokens)
            continue;
        const int64_t at_once = C == 1 ? art_stream::sm_count() : clusters_at_once(C);
        const int64_t rounds = at_once > 0 ? (units + at_once - 1) / at_once : units;
        const int64_t cost = rounds * (slice + (C > 1 ? 8192 : 0));
        if (cost < least) {
            least = cost;
            best = C;
        }
        if (slice <= 4096)
            break;
    }
    return best;
}

// Checks the arguments of a call and lays out its launches; the cluster's size
// is a.cluster.
struct Plan {
    EvictArgs a;
    int64_t units, grid;        // grid: CTAs of the moving kernel
    int smem;                   // of the selection
};

art_status_t plan_of(const art_evict_params_t *p, Plan *pl)
{
    if (!p)
        return ART_ERR_NULL;
    const art_tensor_t &k = p->k_cache, &v = p->v_cache, &pt = p->page_table, &sl = p->seq_lens, &m = p->mass,
                       &ns = p->new_seq_lens, &kp = p->kept;
    if (is_null(&k) || is_null(&v) || is_null(&pt) || is_null(&sl) || is_null(&m) || is_null(&ns) || is_null(&kp))
        return ART_ERR_NULL;
    const art_tensor_t &npt = has(p->new_page_table) ? p->new_page_table : pt;
    const art_tensor_t &nm = has(p->new_mass) ? p->new_mass : m;
    if (k.ndim != 4 || v.ndim != 4 || pt.ndim != 2 || npt.ndim != 2 || sl.ndim != 1 || ns.ndim != 1 || m.ndim != 3 ||
        nm.ndim != 3 || kp.ndim != 3)
        return ART_ERR_SHAPE;
    if ((k.dtype != ART_F32 && k.dtype != ART_BF16) || v.dtype != k.dtype || pt.dtype != ART_I32 || npt.dtype != ART_I32 ||
        sl.dtype != ART_I32 || ns.dtype != ART_I32 || kp.dtype != ART_I32 || m.dtype != ART_F32 || nm.dtype != ART_F32)
        return ART_ERR_DTYPE;
    const int64_t NP = k.shape[0], Hkv = k.shape[1], page = k.shape[2], d = k.shape[3], B = pt.shape[0], mb = pt.shape[1],
                  nb = npt.shape[1], S = mb * page, es = elem_size(k.dtype);
    if (B <= 0 || NP <= 0 || NP > (int64_t)INT32_MAX || Hkv <= 0 || Hkv > 4096 || page <= 0 || page > 4096 || d <= 0 ||
        mb <= 0 || nb <= 0 || B > 65535 || S > (int64_t)INT32_MAX - 4096 || nb * page > (int64_t)INT32_MAX - 4096)
        return ART_ERR_SHAPE;
    for (int i = 0; i < 4; ++i)
        if (v.shape[i] != k.shape[i])
            return ART_ERR_SHAPE;
    if (p->budget < 1 || p->sink < 0 || p->recent < 0 || (int64_t)p->sink + p->recent > p->budget)
        return ART_ERR_PARAM;
    const int64_t most = p->budget < S ? p->budget : S;     // tokens a unit can keep
    if (npt.shape[0] != B || nb * page < most || sl.shape[0] != B || ns.shape[0] != B || m.shape[0] != B ||
        m.shape[1] != Hkv || m.shape[2] < S || nm.shape[0] != B || nm.shape[1] != Hkv || nm.shape[2] < most ||
        kp.shape[0] != B || kp.shape[1] != Hkv || kp.shape[2] != p->budget)
        return ART_ERR_SHAPE;
    for (const art_tensor_t *t : {&k, &v}) {
        if (t->stride[3] != 1 || !aligned(t->data, 16) || (d * es) % 16 || !apart(*t))
            return ART_ERR_SHAPE;
        for (int i = 0; i < 3; ++i)
            if (t->stride[i] <= 0 || (t->stride[i] * es) % 16)
                return ART_ERR_SHAPE;
    }
    if (pt.stride[1] != 1 || pt.stride[0] < 0 || npt.stride[1] != 1 || npt.stride[0] < 0 || sl.stride[0] != 1 ||
        ns.stride[0] != 1 || !aligned(pt.data, 4) || !aligned(npt.data, 4) || !aligned(sl.data, 4) || !aligned(ns.data, 4) ||
        (p->device_status && !aligned(p->device_status, 4)))
        return ART_ERR_SHAPE;
    for (const art_tensor_t *t : {&m, &nm, &kp})
        if (!aligned(t->data, 4) || t->stride[2] != 1 || (B > 1 && t->stride[0] < t->shape[2]) ||
            (Hkv > 1 && t->stride[1] < t->shape[2]))
            return ART_ERR_SHAPE;
    // lengths are read while the new ones are written; weights move in place only onto themselves
    if (ns.data == sl.data || (nm.data == m.data && (nm.stride[0] != m.stride[0] || nm.stride[1] != m.stride[1])))
        return ART_ERR_PARAM;
    if (!apart(nm) || !apart(kp))                            // (m is only read where nm is another tensor)
        return ART_ERR_SHAPE;
    if (S > (int64_t)kMaxCluster * kSliceTokens || d * es > 2048)
        return ART_ERR_UNSUPPORTED;
    EvictArgs &a = pl->a;
    a.k = static_cast<uint8_t *>(k.data);
    a.v = static_cast<uint8_t *>(v.data);
    a.ks0 = k.stride[0] * es;
    a.ks1 = k.stride[1] * es;
    a.ks2 = k.stride[2] * es;
    a.vs0 = v.stride[0] * es;
    a.vs1 = v.stride[1] * es;
    a.vs2 = v.stride[2] * es;
    a.pt = static_cast<const int32_t *>(pt.data);
    a.npt = static_cast<const int32_t *>(npt.data);
    a.pts0 = pt.stride[0];
    a.npts0 = npt.stride[0];
    a.sl = static_cast<const int32_t *>(sl.data);
    a.mass = static_cast<const float *>(m.data);
    a.ms0 = m.stride[0];
    a.ms1 = m.stride[1];
    a.nmass = static_cast<float *>(nm.data);
    a.ns0 = nm.stride[0];
    a.ns1 = nm.stride[1];
    a.nwidth = nm.shape[2];
    a.nsl = static_cast<int32_t *>(ns.data);
    a.kept = static_cast<int32_t *>(kp.data);
    a.kp0 = kp.stride[0];
    a.kp1 = kp.stride[1];
    a.Hkv = (int)Hkv;
    a.page = (int)page;
    a.max_blocks = (int)mb;
    a.num_pages = (int)NP;
    a.budget = p->budget;
    a.sink = p->sink;
    a.recent = p->recent;
    a.in_place = !has(p->new_page_table) || (npt.data == pt.data && npt.stride[0] == pt.stride[0]);
    a.status = p->device_status;
    const int64_t units = B * Hkv;
    const int C = slices_of(S, units);
    a.cluster = C;
    a.row_vecs = (int)(d * es / 16);
    a.lanes = 1;
    const int most_lanes = a.in_place ? kSlideVecs : 32;
    while (a.lanes * 2 <= most_lanes && a.row_vecs % (a.lanes * 2) == 0)
        a.lanes *= 2;
    a.slices = a.row_vecs / a.lanes;
    a.runs = (most + kRunRows - 1) / kRunRows;
    // in place: CTAs for a slice up to four an SM, as far as each still has a run to
    // move (16 units of 131072 to 16384: 93 us, with up to two an SM 120; 64 of 8192
    // to 2048: 44 and 48)
    a.slide_cluster = 1;
    while (a.slide_cluster < kMaxCluster && units * 2 * a.slices * a.slide_cluster * 2 <= 4 * art_stream::sm_count() &&
           a.slide_cluster * kSlideRows < most)
        a.slide_cluster *= 2;
    const int64_t grid = a.in_place ? a.slices * 2 * units * a.slide_cluster : a.runs * units;
    if (units * C > (int64_t)INT32_MAX || grid > (int64_t)INT32_MAX)
        return ART_ERR_SHAPE;
    // One kernel for both steps where few rows move, 128 KB a unit at most: a
    // launch less (one unit of 100 tokens to 50: 5.9 us against 8.1; 64 of 512
    // to 128, 64 KB each, 6.7 against 8.0); with more, one CTA a unit keeps too
    // few copies in flight (256 KB each: 13.0 against 12.1).
    a.whole = !a.in_place && C == 1 && most <= kWholeRows && most * a.row_vecs * 32 <= 128 * 1024;
    pl->units = units;
    pl->grid = grid;
    pl->smem = (int)(((S + C - 1) / C + 31) / 32 * 128);
    return ART_OK;
}

}  // namespace

extern "C" {

int32_t art_evict_cluster_size(const art_evict_params_t *p)
{
    Plan pl;
    const art_status_t st = plan_of(p, &pl);
    return st == ART_OK ? pl.a.cluster : (int32_t)st;
}

art_status_t art_cache_evict(const art_evict_params_t *p, art_stream_t stream)
{
    Plan pl;
    const art_status_t st = plan_of(p, &pl);
    if (st != ART_OK)
        return st;
    const EvictArgs &a = pl.a;
    const int C = a.cluster;
    const auto select = C > 1 ? art_evict_select_kernel<true> : art_evict_select_kernel<false>;
    // (the most that any call needs: another thread's call may stand between this and the launch)
    if (pl.smem > 8 * 1024 &&
        cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, kSliceTokens * 4) != cudaSuccess) {
        cudaGetLastError();
        return ART_ERR_LAUNCH;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = art_stream::launch(select, dim3((unsigned)(pl.units * C)), kSelThreads, pl.smem, s, a, C);
    if (e == cudaSuccess && !a.whole)
        e = art_stream::launch(a.in_place ? art_evict_slide_kernel : art_evict_move_kernel, dim3((unsigned)pl.grid), kMoveThreads, 0,
                               s, a, a.in_place ? a.slide_cluster : 1);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return ART_ERR_LAUNCH;
    }
    return ART_OK;
}

}  // extern "C"
