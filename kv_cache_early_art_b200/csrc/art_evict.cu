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
// weights are read once into the cluster's shared memory; four 8-bit radix
// steps over order-preserving keys, their histograms summed through
// distributed shared memory, give the n-th largest key exactly; a prefix sum
// over the kept flags gives every kept token its row.  No sort, no atomics
// that decide an order: the result is exact and reproducible.
// art_evict_move_kernel copies the kept rows of K and V; bound by HBM, each kept row
// read once and written once.  To new pages all rows move independently.
// In place the rows of a unit move front to back: a CTA owns a column slice
// of one unit's K or V, reads a run of rows into registers and, behind a barrier,
// writes it; since kept[i] >= i, no write reaches a row that a later run
// still has to read, so nothing but that barrier orders it.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/art.h"
#include "art_host.h"

namespace {

namespace cg = cooperative_groups;
using art_host::aligned;
using art_host::elem_size;
using art_host::is_null;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kSliceTokens = 49152;     // weights a CTA holds (192 KB)
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;            // rows a thread has in flight

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
    int B, Hkv, page, max_blocks, new_blocks, num_pages, budget, sink, recent;
    int cluster;
    int in_place;
    // move: 16-byte vectors of a row, of a slice; slices of a row; runs of rows
    int slice_vecs, slices;
    int64_t runs, run_rows;
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
__device__ __forceinline__ uint32_t weight_key(float w)
{
    uint32_t u = __float_as_uint(w);
    if (w != w)
        return 0u;
    if ((u << 1) == 0u)
        u = 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) art_evict_select_kernel(const __grid_constant__ EvictArgs a)
{
    extern __shared__ float w[];                       // this CTA's slice of the weights
    __shared__ uint32_t hist[4][256];
    __shared__ uint32_t all[256];
    __shared__ uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
    __shared__ uint32_t cta_sum[2];
    __shared__ uint32_t found[2];                      // digit, tokens still wanted among its ties
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    const int C = a.cluster, rank = (int)cluster.block_rank();
    const int unit = blockIdx.x / C, b = unit / a.Hkv, h = unit - b * a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = length_of(a, b);
    const int n = L < a.budget ? L : a.budget;
    const float *mrow = a.mass + (int64_t)b * a.ms0 + (int64_t)h * a.ms1;
    float *nrow = a.nmass + (int64_t)b * a.ns0 + (int64_t)h * a.ns1;
    int32_t *krow = a.kept + (int64_t)b * a.kp0 + (int64_t)h * a.kp1;
    const int per = (L + C - 1) / C;
    const int first = min(L, rank * per), count = min(L, first + per) - first;
    if (rank == 0 && h == 0 && tid == 0) {
        a.nsl[b] = n;
        if (a.sl[b] > L)
            report(a.status, ART_ERR_BAD_INDEX);
    }
    for (int i = tid; i < count; i += kSelThreads)
        w[i] = mrow[first + i];
    for (int i = tid; i < 4 * 256; i += kSelThreads)
        hist[i >> 8][i & 255] = 0u;
    __syncthreads();
    auto key_at = [&](int i) -> uint32_t {
        const int t = first + i;
        return t < a.sink || t >= L - a.recent ? 0xffffffffu : weight_key(w[i]);
    };
    uint32_t want = n, prefix = 0u;
    if (n < L) {                                       // the same for the whole cluster
#pragma unroll
        for (int step = 0; step < 4; ++step) {
            const int shift = 24 - 8 * step;
            for (int i = tid; i < count; i += kSelThreads) {
                const uint32_t k = key_at(i);
                if (step == 0 || (k >> (shift + 8)) == prefix)
                    atomicAdd(&hist[step][(k >> shift) & 255u], 1u);
            }
            cluster.sync();
            if (tid < 256) {
                uint32_t s = 0;
                for (int r = 0; r < C; ++r)
                    s += cluster.map_shared_rank(&hist[step][0], r)[tid];
                all[tid] = s;
            }
            __syncthreads();
            if (warp == 0) {
                // lane l holds digits 255 - 8 l down to 248 - 8 l
                uint32_t mine = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    mine += all[255 - 8 * lane - j];
                uint32_t inc = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o)
                        inc += y;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, inc >= want);
                if (lane == __ffs(hit) - 1) {
                    uint32_t above = inc - mine;
                    int d = 255 - 8 * lane;
                    while (above + all[d] < want)
                        above += all[d--];
                    found[0] = (uint32_t)d;
                    found[1] = want - above;
                }
            }
            __syncthreads();
            prefix = (prefix << 8) | found[0];
            want = found[1];
        }
    }
    // prefix: the n-th largest key; `want` of its ties stay, the oldest ones
    const bool every = n == L;
    const int seg = ((count + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int s0 = min(count, warp * seg), s1 = min(count, s0 + seg);
    uint32_t gt = 0, eq = 0;
    for (int i = s0 + lane; i < s1; i += 32) {
        const uint32_t k = key_at(i);
        gt += every || k > prefix;
        eq += !every && k == prefix;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        gt += __shfl_xor_sync(0xffffffffu, gt, o);
        eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    if (lane == 0) {
        warp_gt[warp] = gt;
        warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t sg = 0, se = 0;
        for (int i = 0; i < kSelWarps; ++i) {
            sg += warp_gt[i];
            se += warp_eq[i];
        }
        cta_sum[0] = sg;
        cta_sum[1] = se;
    }
    cluster.sync();
    uint32_t gb = 0, eb = 0;                           // larger keys and ties before this warp's segment
    for (int r = 0; r < rank; ++r) {
        const uint32_t *s = cluster.map_shared_rank(&cta_sum[0], r);
        gb += s[0];
        eb += s[1];
    }
    for (int i = 0; i < warp; ++i) {
        gb += warp_gt[i];
        eb += warp_eq[i];
    }
    cluster.sync();                                    // nobody leaves while its sums are read
    uint32_t at = gb + min(eb, want);
    if (every)
        at = gb;
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = s0; i0 < s1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < s1 ? key_at(i) : 0u;
        const bool tie = i < s1 && !every && k == prefix;
        const unsigned ties = __ballot_sync(0xffffffffu, tie);
        const bool keep = i < s1 && (every || k > prefix || (tie && eb + __popc(ties & below) < want));
        const unsigned keeps = __ballot_sync(0xffffffffu, keep);
        if (keep) {
            const uint32_t pos = at + __popc(keeps & below);
            krow[pos] = first + i;
            nrow[pos] = w[i];
        }
        at += __popc(keeps);
        eb += __popc(ties);
    }
    for (int64_t i = n + rank * kSelThreads + tid; i < a.nwidth; i += C * kSelThreads)
        nrow[i] = 0.f;
    for (int i = n + rank * kSelThreads + tid; i < a.budget; i += C * kSelThreads)
        krow[i] = -1;
}

__global__ void __launch_bounds__(kMoveThreads) art_evict_move_kernel(const __grid_constant__ EvictArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int SV = a.slice_vecs;
    int64_t x = blockIdx.x;
    const int64_t run = x % a.runs;
    x /= a.runs;
    const int slice = (int)(x % a.slices);
    x /= a.slices;
    const bool values = x & 1;
    const int unit = (int)(x >> 1), b = unit / a.Hkv, h = unit - b * a.Hkv;
    const int n = a.nsl[b];
    const int64_t s0 = values ? a.vs0 : a.ks0, s1 = values ? a.vs1 : a.ks1, s2 = values ? a.vs2 : a.ks2;
    const int vec = threadIdx.x % SV, r = threadIdx.x / SV, rows = kMoveThreads / SV;
    uint8_t *base = (values ? a.v : a.k) + (int64_t)h * s1 + ((int64_t)slice * SV + vec) * 16;
    const int32_t *krow = a.kept + (int64_t)b * a.kp0 + (int64_t)h * a.kp1;
    const int32_t *from = a.pt + (int64_t)b * a.pts0, *to = a.npt + (int64_t)b * a.npts0;
    const int64_t lo = run * a.run_rows;
    const int64_t hi = lo + a.run_rows < n ? lo + a.run_rows : n;
    const bool tell = vec == 0 && slice == 0 && !values && h == 0;
    for (int64_t i0 = lo; i0 < hi; i0 += (int64_t)rows * kMoveRows) {
        uint4 d[kMoveRows];
        uint8_t *dst[kMoveRows];
#pragma unroll
        for (int j = 0; j < kMoveRows; ++j) {
            const int64_t i = i0 + r + (int64_t)j * rows;
            dst[j] = nullptr;
            if (i < hi) {
                const int src = krow[i];
                if (a.in_place && src == i)
                    continue;
                const int sp = from[src / a.page], dp = to[i / a.page];
                if (sp < 0 || sp >= a.num_pages || dp < 0 || dp >= a.num_pages) {
                    if (tell)
                        report(a.status, ART_ERR_BAD_INDEX);
                    continue;
                }
                d[j] = *reinterpret_cast<const uint4 *>(base + (int64_t)sp * s0 + (int64_t)(src % a.page) * s2);
                dst[j] = base + (int64_t)dp * s0 + (int64_t)(i % a.page) * s2;
            }
        }
        if (a.in_place)
            __syncthreads();                           // every row of this run is in registers
#pragma unroll
        for (int j = 0; j < kMoveRows; ++j)
            if (dst[j])
                *reinterpret_cast<uint4 *>(dst[j]) = d[j];
    }
}

// --------------------------------------------------------------- host ----

bool has(const art_tensor_t &t) { return t.data != nullptr; }

}  // namespace

extern "C" art_status_t art_cache_evict(const art_evict_params_t *p, art_stream_t stream)
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
        if (t->stride[3] != 1 || !aligned(t->data, 16) || (d * es) % 16)
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
    if (S > (int64_t)kMaxCluster * kSliceTokens || d * es > 2048)
        return ART_ERR_UNSUPPORTED;
    EvictArgs a;
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
    a.B = (int)B;
    a.Hkv = (int)Hkv;
    a.page = (int)page;
    a.max_blocks = (int)mb;
    a.new_blocks = (int)nb;
    a.num_pages = (int)NP;
    a.budget = p->budget;
    a.sink = p->sink;
    a.recent = p->recent;
    a.in_place = !has(p->new_page_table) || (npt.data == pt.data && npt.stride[0] == pt.stride[0]);
    a.status = p->device_status;
    const int64_t units = B * Hkv;
    int C = 1;
    while (C < kMaxCluster && ((S + C - 1) / C > 8192))
        C *= 2;
    a.cluster = C;
    const int64_t rowvecs = d * es / 16;
    int sv = 1;
    const int most_vecs = a.in_place ? 8 : 32;
    while (sv * 2 <= most_vecs && rowvecs % (sv * 2) == 0)
        sv *= 2;
    a.slice_vecs = sv;
    a.slices = (int)(rowvecs / sv);
    const int64_t pass_rows = (int64_t)(kMoveThreads / sv) * kMoveRows;
    a.run_rows = a.in_place ? most : pass_rows;
    a.runs = (most + a.run_rows - 1) / a.run_rows;
    const int64_t grid = a.runs * a.slices * 2 * units;
    if (units * C > (int64_t)INT32_MAX || grid > (int64_t)INT32_MAX)
        return ART_ERR_SHAPE;
    const int smem = (int)((S + C - 1) / C * 4 + 16);
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(art_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return ART_ERR_LAUNCH;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)(units * C));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, art_evict_select_kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return ART_ERR_LAUNCH;
    }
    cudaLaunchConfig_t mc = {};
    cudaLaunchAttribute ma[1];
    mc.gridDim = dim3((unsigned)grid);
    mc.blockDim = dim3(kMoveThreads);
    mc.stream = s;
    ma[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    ma[0].val.programmaticStreamSerializationAllowed = 1;
    mc.attrs = ma;
    mc.numAttrs = 1;
    if (cudaLaunchKernelEx(&mc, art_evict_move_kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return ART_ERR_LAUNCH;
    }
    return ART_OK;
}
