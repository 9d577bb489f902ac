// art_split.cu -- exact single-token decode attention over the paged cache,
// split over the cache's length and joined (art_decode_attention_split in
// art.h), with each cached token's attention weight added up on request.
//
// For query head i of sequence b (kv-head h = i / G) over the L_b cached rows
//     x_t = sm_scale q_i . k_t,   o = sum_t exp(x_t - lse) v_t,   lse = log sum_t exp(x_t),
// and with `mass`  mass[b, h, t] += sum over the G heads of exp(x_t - lse).
//
// What bounds it: the cache is read once (2 L d elements per kv-head) and each
// byte meets 2 G multiply-adds, G <= 8: HBM, never the arithmetic, so the
// products run on mma.sync from tiles of 16 tokens x 8 heads and the
// design is about keeping loads in flight on every SM until the end.
//
// Split: all tiles (16 or 8 tokens) of all (sequence, kv-head) units form one list;
// CTA c of n takes the c-th n-th of it, whatever the lengths are (they are
// only known on the device).  A unit inside one CTA's share is finished there;
// one that several CTAs share leaves (max, sum, unnormalised output) of each
// part in the workspace and a second kernel, launched as a programmatic
// dependent, joins them.  (Short units, and few of them, are attended by a
// cluster of CTAs each, which join their parts through distributed shared
// memory: one kernel, no workspace.)  Nothing is carried from call to call and no atomics
// decide a result, so equal inputs give equal bits.
//
// Inside a CTA the warps take the tiles in turn and never wait for one another
// except at a unit's end: each fills its own ring of tiles with 16-byte
// asynchronous copies (rows are looked up in the page table one by one, so any
// page size works; the 16-byte pieces of a row are XOR-swizzled against bank
// conflicts), keeps its own running maximum, sum and output in registers, and
// rescales them only when a maximum grew.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/art.h"
#include "art_host.h"
#include "art_ptx.cuh"
#include "art_stream.cuh"

namespace {

using namespace art;
namespace cg = cooperative_groups;
using art_stream::follow;
using art_stream::lead;
using art_host::aligned;
using art_host::apart;
using art_host::elem_size;
using art_host::is_null;

// Tokens a warp handles at a time: the matrix instruction's 16 rows; on fp32
// caches eight where 16 would leave room for too few warps.  Measured, 16 and 8
// tokens, share of the copy rate: d = 256 39-60 % and 46-85 %, d = 128 with up
// to four heads a kv-head 77-80 and 87-91, with eight 60 and 58, d = 64 64-88 and
// 52-71.
template <typename T, int D, int GP>
constexpr int kTileOf = sizeof(T) == 4 && (D == 256 || (D == 128 && GP <= 4)) ? 8 : 16;
constexpr int kMaxG = 8;
constexpr int kMaxCluster = 8;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr double kLog2e = 1.4426950408889634;

struct SplitArgs {
    const void *q;
    int64_t qs0, qs1;
    const void *k, *v;
    int64_t ks0, ks1, ks2, vs0, vs1, vs2;   // page, head, token strides (bytes)
    const int32_t *pt;
    int64_t pts0;
    const int32_t *sl;
    void *out;
    int64_t os0, os1;
    int out_bf16;
    float *lse;
    int64_t ls0, ls1;
    float *mass;
    int64_t ms0, ms1;
    int B, Hq, Hkv, G, page, max_blocks, num_pages;
    int page_whole;               // the page is a multiple of the tile
    int tile_log;                 // log2 of the tile's tokens
    float scale_log2;
    int32_t *status;
    int ctas, least;              // CTAs launched; fewest tiles worth one (see sharers)
    int cluster;                  // CTAs on a unit, or 0: the tiles are shared out evenly
    int join_x, join_heads;       // CTAs that join a unit, heads each of them takes
    // workspace: parts [ctas][2] of max [8], sum [8], output [G][D]; finished units' max and sum [units][G],
    // products q.k [units][max_tokens][G] (with mass only)
    float *parts;
    float2 *unit_sum;
    float *logits;
    int64_t max_tokens;
};

// A softmax weight, exp(sm_scale (x - m)), of a product x = q.k at the largest
// product m (0 where there is none: -inf and infinities then give 0 and NaN as
// they should).  The maxima are held as products, unscaled: their difference is
// small where the weight counts, so it is rounded to that size, and a maximum's
// own weight is 1 however large it is.  (Held scaled and rounded, they left the
// rounding in the exponent: a weight of 2^-64 or 2^64 for logits of 2^30.)
__device__ __forceinline__ float weight(const SplitArgs &a, float x, float m) { return ex2_approx((x - m) * a.scale_log2); }
__device__ __forceinline__ float or_zero(float m) { return m == -CUDART_INF_F ? 0.f : m; }
// log sum exp of a maximum and a sum at it, natural units; -inf of nothing
__device__ __forceinline__ float lse_of(const SplitArgs &a, float m, float l)
{
    return l > 0.f || l != l ? fmaf(m, a.scale_log2, log2f(l)) * kLn2 : -CUDART_INF_F;
}

__host__ __device__ inline int64_t part_floats(int64_t G, int64_t D) { return 2 * kMaxG + G * D; }

__device__ __forceinline__ void report(int32_t *status, int32_t code)
{
    if (status)
        atomicCAS(status, 0, code);
}

// rows of sequence b that the page table can hold
__device__ __forceinline__ int length_of(const SplitArgs &a, int b)
{
    const int64_t cap = (int64_t)a.max_blocks * a.page;
    const int L = __ldcg(a.sl + b);
    return L <= 0 ? 0 : (int)(L < cap ? L : cap);
}

__device__ __forceinline__ int tiles_of(const SplitArgs &a, int L) { return (L + (1 << a.tile_log) - 1) >> a.tile_log; }

// Lanes b0 .. b0 + 31 of the batch: lane's sequence length and the inclusive
// prefix of the tiles one kv-head has there, by one warp.
struct Chunk {
    int L;
    uint32_t inc;
};
__device__ __forceinline__ Chunk chunk_of(const SplitArgs &a, int b0, int lane)
{
    Chunk c;
    c.L = b0 + lane < a.B ? length_of(a, b0 + lane) : 0;
    c.inc = (uint32_t)tiles_of(a, c.L);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, c.inc, o);
        if (lane >= o)
            c.inc += y;
    }
    return c;
}

// tiles of the whole batch (under 2^31: the host sees to it), by one warp;
// first: the first chunk
__device__ __forceinline__ int batch_tiles(const SplitArgs &a, const Chunk &first, int lane)
{
    int n = __shfl_sync(0xffffffffu, first.inc, 31);
    for (int b0 = 32; b0 < a.B; b0 += 32)
        n += __shfl_sync(0xffffffffu, chunk_of(a, b0, lane).inc, 31);
    return n * a.Hkv;
}

// CTAs that share the list of `total` tiles: a share is a whole number of
// rounds of the CTA's warps, no smaller than pays for its part of the join
// (`least` tiles, 64 tokens; twice that where a unit has no more than that, or
// a tile is large).  Measured: 4 units of 1024 tokens 6.5 us in shares of 64
// and 7.6 in 128; 4 units of 100 tokens 7.5 and 5.3; a unit of 8192 tokens of d
// = 256 12.9 and 12.1.
__device__ __forceinline__ int sharers(const SplitArgs &a, int total)
{
    int share = total / a.ctas + (total % a.ctas != 0);
    if (share > 3 * (64 >> a.tile_log))
        return a.ctas;
    const int few = 128 >> a.tile_log;
    const int least = total <= few * a.B * a.Hkv && a.least < few ? few : a.least;
    share = share < least ? least : (share + 3) & ~3;
    return total > 0 ? (total + share - 1) / share : 1;
}

__device__ __forceinline__ int share_begin(int total, int c, int n) { return (int)((int64_t)total * c / n); }

// the CTA whose share holds tile x
__device__ __forceinline__ int share_of(int x, int total, int n)
{
    // (a 32-bit division, where it fits, is a fraction of a 64-bit one's latency)
    if (total <= 0x7fffffff / n)
        return (int)((((uint32_t)x + 1u) * (uint32_t)n - 1u) / (uint32_t)total);
    return (int)((((int64_t)x + 1) * n - 1) / total);
}

// A place in the list: tile s of unit (b, h), nt tiles and L rows there.
struct Place {
    int b, h, s, nt, L;
};

// Finds tile x of the list, by one warp (x < total).
__device__ __forceinline__ Place find_tile(const SplitArgs &a, int x, Chunk k, int lane)
{
    for (int b0 = 0;;) {
        const unsigned hit = __ballot_sync(0xffffffffu, (int)k.inc * a.Hkv > x);
        if (hit || b0 + 32 >= a.B) {
            const int src = hit ? __ffs(hit) - 1 : 31;
            Place p;
            p.b = b0 + src;
            p.L = __shfl_sync(0xffffffffu, k.L, src);
            p.nt = tiles_of(a, p.L);
            const int in = x - ((int)__shfl_sync(0xffffffffu, k.inc, src) - p.nt) * a.Hkv;
            p.h = p.nt ? in / p.nt : 0;
            p.s = in - p.h * p.nt;
            return p;
        }
        x -= (int)__shfl_sync(0xffffffffu, k.inc, 31) * a.Hkv;
        b0 += 32;
        k = chunk_of(a, b0, lane);
    }
}

// Moves a place on by n tiles of the list; stays in range while the caller's count does.
__device__ __forceinline__ void advance(const SplitArgs &a, Place &p, int n)
{
    p.s += n;
    while (p.s >= p.nt) {
        p.s -= p.nt;
        if (++p.h == a.Hkv) {
            p.h = 0;
            do {
                if (++p.b >= a.B) {                       // past the list: only reached by a cursor that ends here
                    p.b = a.B - 1;
                    p.nt = 0x7fffffff;
                    return;
                }
                p.L = length_of(a, p.b);
                p.nt = tiles_of(a, p.L);
            } while (p.nt == 0);
        }
    }
}

// The cache streams through once: evict_first keeps it from pushing the parts,
// the logits and the caller's data out of L2.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid, uint64_t once)
{
    const int n = valid ? 16 : 0;   // 0: the 16 bytes are zeroed, nothing is read
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(n), "l"(once)
                 : "memory");
}
__device__ __forceinline__ uint64_t evict_first()
{
    uint64_t policy;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One warp requests tile (b, h, s): its rows of K and of V into ring slot
// `dst` (K rows, then V rows; 16-byte piece i of row r sits at i ^ (r & 7)).
// Rows past the sequence, or in a page outside the cache, are zeroed and left
// out of the returned row mask.  Where the page is a multiple of the tile
// (page_whole) the tile lies in one page and its rows are one stride apart;
// else each row is looked up (measured at d = 256, 32-row pages: the look-up
// of every row took 400 of a tile's 1600 instructions and 40 % of the time).
template <typename T, int D, int TT>
__device__ __forceinline__ unsigned load_tile(const SplitArgs &a, const Place &p, uint32_t dst, uint64_t once, int lane)
{
    constexpr int RB = D * (int)sizeof(T);               // bytes of a row
    constexpr int CH = RB / 16;                          // 16-byte pieces of a row: 8 .. 64
    constexpr int LPR = CH < 32 ? CH : 32;               // lanes on one row
    constexpr int RPI = 32 / LPR;                        // rows per instruction
    constexpr int PPL = CH / LPR;                        // pieces per lane and row
    const int t0 = p.s * TT;
    const int32_t *row = a.pt + (int64_t)p.b * a.pts0;
    const int r0 = lane / LPR, c0 = lane % LPR;
    const char *kh = static_cast<const char *>(a.k) + (int64_t)p.h * a.ks1 + c0 * 16;
    const char *vh = static_cast<const char *>(a.v) + (int64_t)p.h * a.vs1 + c0 * 16;
    if (a.page_whole) {
        const int blk = t0 / a.page, off = t0 - blk * a.page;
        const int pg = row[blk];
        const bool ok = pg >= 0 && pg < a.num_pages;
        if (!ok && lane == 0)
            report(a.status, ART_ERR_BAD_INDEX);
        const int rows = ok ? min(TT, p.L - t0) : 0;
        const int at = ok ? pg : 0;
        const char *ks = kh + at * a.ks0 + (int64_t)(off + r0) * a.ks2;
        const char *vs = vh + at * a.vs0 + (int64_t)(off + r0) * a.vs2;
#pragma unroll
        for (int i = 0; i < TT / RPI; ++i) {
            const int r = r0 + i * RPI;
#pragma unroll
            for (int j = 0; j < PPL; ++j) {
                const uint32_t to = dst + r * RB + (((c0 + j * LPR) ^ (r & 7)) * 16);
                cp_async16(to, ks + j * LPR * 16, r < rows, once);
                cp_async16(to + TT * RB, vs + j * LPR * 16, r < rows, once);
            }
            ks += RPI * a.ks2;
            vs += RPI * a.vs2;
        }
        return (1u << rows) - 1u;
    }
    int pg = 0, off = 0;
    bool ok = false;
    if (lane < TT && t0 + lane < p.L) {
        const int t = t0 + lane;
        const int blk = t / a.page;
        off = t - blk * a.page;
        pg = row[blk];
        ok = pg >= 0 && pg < a.num_pages;
        if (!ok) {
            report(a.status, ART_ERR_BAD_INDEX);
            pg = off = 0;
        }
    }
    const unsigned mask = __ballot_sync(0xffffffffu, ok);
#pragma unroll
    for (int i = 0; i < TT / RPI; ++i) {
        const int r = r0 + i * RPI;
        const int64_t rp = __shfl_sync(0xffffffffu, pg, r), ro = __shfl_sync(0xffffffffu, off, r);
        const bool v = (mask >> r) & 1;
        const char *ks = kh + rp * a.ks0 + ro * a.ks2, *vs = vh + rp * a.vs0 + ro * a.vs2;
#pragma unroll
        for (int j = 0; j < PPL; ++j) {
            const uint32_t to = dst + r * RB + (((c0 + j * LPR) ^ (r & 7)) * 16);
            cp_async16(to, ks + j * LPR * 16, v, once);
            cp_async16(to + TT * RB, vs + j * LPR * 16, v, once);
        }
    }
    return mask;
}

// D = A(16x16, row) * B(16x8, col), bf16 inputs, fp32 sums
__device__ __forceinline__ void mma_from_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// ---- one warp's running state over its tiles of a unit ----------------------

// bf16: S^T = K q^T (16 tokens x 8 heads), O^T += V^T P with mma.m16n8k16.  P
// enters as the sum of three bf16 terms, all its 24 bits: with two the output
// was 1.2e-6 off at 131072 tokens, with three 4.4e-7, at the same time (the
// products hide behind the loads).  SHARED (G <= 4): the heads are held twice,
// columns 4-7 repeat 0-3, so that one product takes two of the terms.
template <int D, bool SHARED>
struct TensorState {
    static constexpr int KS = D / 16;
    uint32_t qb[KS][2];
    float o[KS][4];
    float m[2], l[2];             // heads 2c, 2c + 1; l: this lane's tokens only
    int r, c;

    __device__ __forceinline__ void begin(const SplitArgs &a, int b, int h, int lane, const float *)
    {
        r = lane >> 2;
        c = lane & 3;
        const int row = SHARED ? (r & 3) : r;
        const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q) + (int64_t)b * a.qs0 +
                                  (int64_t)(h * a.G + row) * a.qs1 + 2 * c;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            qb[ks][0] = qb[ks][1] = 0u;
            if (row < a.G) {
                qb[ks][0] = *reinterpret_cast<const uint32_t *>(qp + ks * 16);
                qb[ks][1] = *reinterpret_cast<const uint32_t *>(qp + ks * 16 + 8);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[ks][i] = 0.f;
        }
        m[0] = m[1] = -CUDART_INF_F;
        l[0] = l[1] = 0.f;
    }

    __device__ __forceinline__ void tile(const SplitArgs &a, uint32_t kt, unsigned mask, int rows, float *logits, float *, int lane)
    {
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
        // the ring's slots are aligned to their rows: piece 2 ks of a row is an XOR away
        const uint32_t ka = kt + (lane & 15) * (D * 2) + (((lane >> 4) ^ (lane & 7)) * 16);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t a0, a1, a2, a3;
            ldmatrix_x4(ka ^ (ks * 32), a0, a1, a2, a3);
            mma_bf16_16816((ks & 1) ? s2 : s, a0, a1, a2, a3, qb[ks][0], qb[ks][1]);
        }
        const bool v0 = (mask >> r) & 1, v1 = (mask >> (r + 8)) & 1;
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = ((i >> 1) ? v1 : v0) ? s[i] + s2[i] : -CUDART_INF_F;
        if (logits) {
            const int g = 2 * c;
            if (g < a.G) {
                if (r < rows)
                    logits[r * a.G + g] = x[0];
                if (r + 8 < rows)
                    logits[(r + 8) * a.G + g] = x[2];
            }
            if (g + 1 < a.G) {
                if (r < rows)
                    logits[r * a.G + g + 1] = x[1];
                if (r + 8 < rows)
                    logits[(r + 8) * a.G + g + 1] = x[3];
            }
        }
        float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
        }
        if (__any_sync(0xffffffffu, mx0 > m[0] || mx1 > m[1])) {
            const float n0 = fmaxf(m[0], mx0), n1 = fmaxf(m[1], mx1);
            const float f0 = m[0] == n0 ? 1.f : weight(a, m[0], n0), f1 = m[1] == n1 ? 1.f : weight(a, m[1], n1);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                o[ks][0] *= f0;
                o[ks][1] *= f1;
                o[ks][2] *= f0;
                o[ks][3] *= f1;
            }
            l[0] *= f0;
            l[1] *= f1;
            m[0] = n0;
            m[1] = n1;
        }
        float p[4];
        const uint64_t one = pk2(1.f, 1.f), scale = pk2(a.scale_log2, a.scale_log2), off = pk2(-or_zero(m[0]), -or_zero(m[1]));
#pragma unroll
        for (int i = 0; i < 4; i += 2) {                 // weight() of both heads at a time
            const uint64_t e = mul2(fma2(pk2(x[i], x[i + 1]), one, off), scale);
            p[i] = ex2_approx(lo2(e));
            p[i + 1] = ex2_approx(hi2(e));
        }
        l[0] += p[0] + p[2];
        l[1] += p[1] + p[3];
        uint32_t bh[2], bl[2], br[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const __nv_bfloat162 hi = __floats2bfloat162_rn(p[2 * half], p[2 * half + 1]);
            const float2 hf = __bfloat1622float2(hi);
            const float r0 = p[2 * half] - hf.x, r1 = p[2 * half + 1] - hf.y;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(r0, r1);
            const float2 lf = __bfloat1622float2(lo);
            const __nv_bfloat162 rest = __floats2bfloat162_rn(r0 - lf.x, r1 - lf.y);
            const uint32_t hu = *reinterpret_cast<const uint32_t *>(&hi), lu = *reinterpret_cast<const uint32_t *>(&lo),
                           ru = *reinterpret_cast<const uint32_t *>(&rest);
            if constexpr (SHARED) {
                bh[half] = movmatrix_trans(c < 2 ? hu : lu);
                br[half] = movmatrix_trans(c < 2 ? ru : 0u);
                bl[half] = 0u;
            } else {
                bh[half] = movmatrix_trans(hu);
                bl[half] = movmatrix_trans(lu);
                br[half] = movmatrix_trans(ru);
            }
        }
        const uint32_t va = kt + 16 * D * 2 + ((lane & 7) + (lane >> 4) * 8) * (D * 2) +
                            ((((lane >> 3) & 1) ^ (lane & 7)) * 16);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t a0, a1, a2, a3;
            ldmatrix_x4_trans(va ^ (ks * 32), a0, a1, a2, a3);
            // a tile's sum starts at zero and joins the output by an ordinary
            // addition: the matrix unit truncates, and along a long cache those
            // errors add up one way (4.5e-6 of the output at 131072 tokens)
            float t[4];
            mma_from_zero(t, a0, a1, a2, a3, bh[0], bh[1]);
            if constexpr (!SHARED)
                mma_bf16_16816(t, a0, a1, a2, a3, bl[0], bl[1]);
            mma_bf16_16816(t, a0, a1, a2, a3, br[0], br[1]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[ks][i] += t[i];
        }
    }

    // writes this warp's part: ml [2][kMaxG] (max, sum), po [G][D]
    __device__ __forceinline__ void end(const SplitArgs &a, float *ml, float *po, int)
    {
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], off);
        }
        if (r == 0) {
            ml[2 * c] = m[0];
            ml[2 * c + 1] = m[1];
            ml[kMaxG + 2 * c] = l[0];
            ml[kMaxG + 2 * c + 1] = l[1];
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            float t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                t[i] = o[ks][i];
                if constexpr (SHARED)
                    t[i] += __shfl_xor_sync(0xffffffffu, o[ks][i], 2);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int g = 2 * c + (i & 1), d = ks * 16 + r + (i >> 1) * 8;
                if (g < a.G)
                    po[g * D + d] = t[i];
            }
        }
    }
};

// fp32: CUDA cores.  Scores: lane (token, every second or fourth 16-byte piece), all heads, K
// pieces from the ring and q broadcast from shared memory; output: each lane
// owns 16-byte columns of V and takes the weights from shared memory.  Both in
// packed pairs (two multiply-adds an instruction).
template <int D, int GP>
struct ScalarState {
    static constexpr int TT = kTileOf<float, D, GP>;     // tokens
    static constexpr int NP = 32 / TT;                   // lanes on each
    static constexpr int CH = D / 4;                     // 16-byte columns
    static constexpr int LPR = CH < 32 ? CH : 32;
    static constexpr int PPL = CH / LPR;
    static constexpr int RPI = 32 / LPR;                 // lanes that share a column take alternate tokens
    uint64_t o[PPL][GP][2];                              // packed pairs
    float m[GP], l[GP];                                  // l: this lane's token only
    const float *q;                                      // [GP][D] in shared memory (zeros past G)

    __device__ __forceinline__ void begin(const SplitArgs &, int, int, int, const float *qs)
    {
        q = qs;
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            m[g] = -CUDART_INF_F;
            l[g] = 0.f;
#pragma unroll
            for (int j = 0; j < PPL; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    o[j][g][e] = 0ull;
        }
    }

    __device__ __forceinline__ void tile(const SplitArgs &a, uint32_t kt, unsigned mask, int rows, float *logits, float *ps, int lane)
    {
        const ulonglong2 *kb = reinterpret_cast<const ulonglong2 *>(__cvta_shared_to_generic(kt));
        const int t = lane % TT, part = lane / TT;
        // four sums a head and lane: short chains of roundings (with one over
        // half a row, outputs at d = 256 were up to 1.6e-6 off)
        uint64_t s4[GP][2];
        float s[GP];
#pragma unroll
        for (int g = 0; g < GP; ++g)
            s4[g][0] = s4[g][1] = 0ull;
#pragma unroll 4
        for (int i = 0; i < CH / NP; ++i) {
            const int ch = NP * i + part;                // (q's pieces side by side: no bank conflict)
            const ulonglong2 kv = kb[t * CH + (ch ^ (t & 7))];
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                const ulonglong2 qv = *reinterpret_cast<const ulonglong2 *>(q + g * D + ch * 4);
                s4[g][0] = fma2(kv.x, qv.x, s4[g][0]);
                s4[g][1] = fma2(kv.y, qv.y, s4[g][1]);
            }
        }
#pragma unroll
        for (int g = 0; g < GP; ++g)
            s[g] = (lo2(s4[g][0]) + hi2(s4[g][0])) + (lo2(s4[g][1]) + hi2(s4[g][1]));
        const bool v = (mask >> t) & 1;
        bool grew = false;
        float mx[GP];
#pragma unroll
        for (int g = 0; g < GP; ++g) {
#pragma unroll
            for (int off = TT; off < 32; off <<= 1)
                s[g] += __shfl_xor_sync(0xffffffffu, s[g], off);
            s[g] = v ? s[g] : -CUDART_INF_F;
            if (logits && part == 0 && t < rows && g < a.G)
                logits[t * a.G + g] = s[g];
            mx[g] = s[g];
#pragma unroll
            for (int off = 1; off < TT; off <<= 1)
                mx[g] = fmaxf(mx[g], __shfl_xor_sync(0xffffffffu, mx[g], off));
            grew = grew || mx[g] > m[g];
        }
        if (grew) {                                      // the same on every lane
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                const float n = fmaxf(m[g], mx[g]);
                const float f = m[g] == n ? 1.f : weight(a, m[g], n);
                m[g] = n;
                l[g] *= f;
                const uint64_t ff = pk2(f, f);
#pragma unroll
                for (int j = 0; j < PPL; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        o[j][g][e] = mul2(o[j][g][e], ff);
            }
        }
        const uint64_t one = pk2(1.f, 1.f), scale = pk2(a.scale_log2, a.scale_log2);
#pragma unroll
        for (int g = 0; g < GP; g += 2) {                // weight() of two heads at a time (123.4 us; 125.5 one by one)
            const uint64_t e = mul2(fma2(pk2(s[g], s[g + 1]), one, pk2(-or_zero(m[g]), -or_zero(m[g + 1]))), scale);
            const float p0 = ex2_approx(lo2(e)), p1 = ex2_approx(hi2(e));
            if (part == 0) {
                l[g] += p0;
                l[g + 1] += p1;
                ps[t * GP + g] = p0;
                ps[t * GP + g + 1] = p1;
            }
        }
        __syncwarp();
        const ulonglong2 *vb = kb + TT * CH;
        const int c0 = lane % LPR, sub = lane / LPR;
#pragma unroll 4
        for (int i = 0; i < TT / RPI; ++i) {
            const int tt = i * RPI + sub;
            float pg[GP];
#pragma unroll
            for (int g = 0; g < GP; g += 4)
                *reinterpret_cast<float4 *>(pg + g) = *reinterpret_cast<const float4 *>(ps + tt * GP + g);
#pragma unroll
            for (int j = 0; j < PPL; ++j) {
                const int ch = c0 + j * LPR;
                const ulonglong2 vv = vb[tt * CH + (ch ^ (tt & 7))];
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const uint64_t pp = pk2(pg[g], pg[g]);
                    o[j][g][0] = fma2(pp, vv.x, o[j][g][0]);
                    o[j][g][1] = fma2(pp, vv.y, o[j][g][1]);
                }
            }
        }
        __syncwarp();                                    // ps is rewritten by the next tile
    }

    __device__ __forceinline__ void end(const SplitArgs &a, float *ml, float *po, int lane)
    {
        const int c0 = lane % LPR, sub = lane / LPR;
#pragma unroll
        for (int g = 0; g < GP; ++g) {
#pragma unroll
            for (int off = 16; off; off >>= 1)
                l[g] += __shfl_xor_sync(0xffffffffu, l[g], off);
            if (lane == 0) {
                ml[g] = m[g];
                ml[kMaxG + g] = l[g];
            }
#pragma unroll
            for (int j = 0; j < PPL; ++j) {
                float4 t;
                float *tv = &t.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    tv[e] = e & 1 ? hi2(o[j][g][e >> 1]) : lo2(o[j][g][e >> 1]);
#pragma unroll
                    for (int off = LPR; off < 32; off <<= 1)
                        tv[e] += __shfl_xor_sync(0xffffffffu, tv[e], off);
                }
                if (sub == 0 && g < a.G)
                    *reinterpret_cast<float4 *>(po + g * D + (c0 + j * LPR) * 4) = t;
            }
        }
    }
};

template <typename T, int D, int GP>
struct StateOf {
    using type = TensorState<D, (GP <= 4)>;
};
template <int D, int GP>
struct StateOf<float, D, GP> {
    using type = ScalarState<D, GP>;
};

// shape of the kernel for a row of D elements and up to GP heads
template <typename T, int D, int GP>
struct Shape {
    static constexpr bool f32 = std::is_same<T, float>::value;
    static constexpr int rows = kTileOf<T, D, GP>;                      // of a tile
    static constexpr int tile_bytes = 2 * rows * D * (int)sizeof(T);    // 4, 8 or 16 KB
    static constexpr int stages = tile_bytes <= 4096 ? 6 : 3;           // ring slots a warp
    static constexpr int warps = f32 && D == 256 && GP > 4 ? 3 : 4;     // (a fourth one's ring and part do not fit)
    static constexpr int ctas_per_sm = tile_bytes > 8192 ? 1 : 2;
    // most tiles of a CTA of a cluster (their logits are held in what shared memory is left)
    static constexpr int part_tiles = rows == 8 ? 16 : !f32 && D == 256 && GP > 4 ? 4 : 8;
    // rings; one part of a unit a warp; the fp32 path's weights and queries
    static constexpr int ring_bytes = warps * stages * tile_bytes;
    static constexpr int smem =
        ring_bytes + warps * (2 * kMaxG + GP * D) * 4 + (f32 ? (warps * rows * GP + GP * D) * 4 : 0);
    // and with clusters the CTA's max and sum, and its logits
    static constexpr int smem_cluster = smem + 2 * kMaxG * 4 + part_tiles * rows * GP * 4;
    static_assert(smem_cluster <= 227 * 1024, "a CTA an SM");
    static_assert(ctas_per_sm * (smem + 1024) <= 228 * 1024, "CTAs an SM");
};

__device__ __forceinline__ void store_out(const SplitArgs &a, int b, int i, int d, float v)
{
    const int64_t at = (int64_t)b * a.os0 + (int64_t)i * a.os1 + d;
    if (a.out_bf16)
        static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(a.out)[at] = v;
}

// The end of a unit that a cluster attended: the CTA's warps are joined in its
// shared memory, the cluster's parts through distributed shared memory, and
// every CTA writes a slice of the output and adds its own tokens' weights.
template <typename T, int D, int GP>
__device__ __forceinline__ void join_cluster(const SplitArgs &a, const Place &cur, int at, int end, int C, int rank,
                                             float *ml, float *po, float *cm, const float *logits)
{
    using S = Shape<T, D, GP>;
    constexpr int NW = S::warps, TT = S::rows;
    const int n = a.G * D;                               // cm [2][kMaxG]: the CTA's max and sum; its output goes to po
    for (int i = threadIdx.x; i < n; i += NW * 32) {
        const int g = i / D;
        float mm = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < NW; ++w)
            mm = fmaxf(mm, ml[w * 2 * kMaxG + g]);
        const float base = or_zero(mm);
        float ll = 0.f, oo = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = weight(a, ml[w * 2 * kMaxG + g], base);
            ll = fmaf(f, ml[w * 2 * kMaxG + kMaxG + g], ll);
            oo = fmaf(f, po[w * GP * D + i], oo);
        }
        po[i] = oo;                                      // this thread alone reads place i
        if (i == g * D) {
            cm[g] = mm;
            cm[kMaxG + g] = ll;
        }
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (C > 1)
        cluster.sync();
    else
        __syncthreads();
    // max and sum of head g over the cluster
    auto whole = [&](int g, float (&f)[kMaxCluster], float &mm, float &ll) {
        float pm[kMaxCluster], pl[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
            pm[r] = -CUDART_INF_F;
            pl[r] = 0.f;
            if (r < C) {
                const float *p = C > 1 ? cluster.map_shared_rank(cm, r) : cm;
                pm[r] = p[g];
                pl[r] = p[kMaxG + g];
            }
        }
        mm = -CUDART_INF_F;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            mm = fmaxf(mm, pm[r]);
        ll = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
            f[r] = weight(a, pm[r], or_zero(mm));
            ll = fmaf(f[r], pl[r], ll);
        }
    };
    for (int i = n * rank / C + threadIdx.x; i < n * (rank + 1) / C; i += NW * 32) {
        const int g = i / D, d = i - g * D, head = cur.h * a.G + g;
        float o[kMaxCluster], f[kMaxCluster], mm, ll;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            o[r] = r < C ? (C > 1 ? cluster.map_shared_rank(po, r) : po)[i] : 0.f;
        whole(g, f, mm, ll);
        float oo = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            oo = fmaf(f[r], o[r], oo);
        const bool some = ll > 0.f || ll != ll;
        store_out(a, cur.b, head, d, some ? oo / ll : 0.f);
        if (d == 0 && a.lse)
            a.lse[(int64_t)cur.b * a.ls0 + (int64_t)head * a.ls1] = lse_of(a, mm, ll);
    }
    if (a.mass) {
        if (threadIdx.x < a.G) {
            float f[kMaxCluster], mm, ll;
            whole(threadIdx.x, f, mm, ll);
            ml[threadIdx.x] = or_zero(mm);                       // (the warps' maxima are joined)
            ml[kMaxG + threadIdx.x] = ll == 0.f ? 0.f : log2f(ll);
        }
        __syncthreads();
        const int t0 = at * TT;
        float *mrow = a.mass + (int64_t)cur.b * a.ms0 + (int64_t)cur.h * a.ms1;
        const int upto = cur.L < end * TT ? cur.L : end * TT;
        for (int t = t0 + threadIdx.x; t < upto; t += NW * 32) {
            float w = 0.f;
            for (int g = 0; g < a.G; ++g)
                w += ex2_approx(fmaf(logits[(t - t0) * a.G + g] - ml[g], a.scale_log2, -ml[kMaxG + g]));
            mrow[t] += w;
        }
    }
    if (C > 1)
        cluster.sync();                                  // nobody leaves while its part is read
}

// SMALL: a cluster of a.cluster CTAs attends a whole unit, a part each, and
// joins the parts through distributed shared memory; see the host side.
template <typename T, int D, int GP, bool SMALL>
__global__ void __launch_bounds__(Shape<T, D, GP>::warps * 32, Shape<T, D, GP>::ctas_per_sm)
    art_split_kernel(const __grid_constant__ SplitArgs a)
{
    using S = Shape<T, D, GP>;
    constexpr int NW = S::warps, ST = S::stages, TT = S::rows;
    extern __shared__ __align__(1024) uint8_t smem[];
    follow();
    if constexpr (!SMALL)
        lead();                                          // the joining kernel
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *ml = reinterpret_cast<float *>(smem + S::ring_bytes);                // [NW][2][kMaxG]
    float *po = ml + NW * 2 * kMaxG;                                        // [NW][GP][D]
    float *ps = po + NW * GP * D;                                           // fp32: [NW][TT][GP]
    float *qs = ps + NW * TT * GP;                                          // fp32: [GP][D]
    float *cm = reinterpret_cast<float *>(smem + S::smem);                  // SMALL: [2][kMaxG], logits
    const uint32_t ring = smem_u32(smem) + warp * ST * S::tile_bytes;

    int at, end;                                         // this CTA's tiles
    Place cur;                                           // the segment being attended
    int cta = blockIdx.x, C = 1, rank = 0;
    if constexpr (SMALL) {
        C = a.cluster;
        const int u = cta / C;
        rank = cta - u * C;
        cur.b = u / a.Hkv;
        cur.h = u - cur.b * a.Hkv;
        cur.L = length_of(a, cur.b);
        cur.nt = tiles_of(a, cur.L);
        if (cur.h == 0 && rank == 0 && threadIdx.x == 0 && a.sl[cur.b] > cur.L)
            report(a.status, ART_ERR_BAD_INDEX);
        at = cur.s = cur.nt * rank / C;                  // places within the unit
        end = cur.nt * (rank + 1) / C;
    } else {
        const Chunk chunk = chunk_of(a, 0, lane);
        const int total = batch_tiles(a, chunk, lane);
        const int n = sharers(a, total);
        if (total == 0 || cta >= n)
            return;
        at = share_begin(total, cta, n);
        end = share_begin(total, cta + 1, n);
        if (at >= end)
            return;
        cur = find_tile(a, at, chunk, lane);
    }
    // this warp's tiles: at + warp, at + warp + NW, ...; `next` is the one to request
    Place next = cur;
    int next_at = at + warp;
    if (next_at < end)
        advance(a, next, warp);
    unsigned masks[ST];
#pragma unroll
    for (int i = 0; i < ST; ++i)
        masks[i] = 0u;
    const uint64_t once = evict_first();
    auto request = [&](int slot) -> unsigned {
        unsigned mk = 0u;
        if (next_at < end) {
            mk = load_tile<T, D, TT>(a, next, ring + slot * S::tile_bytes, once, lane);
            next_at += NW;
            if (next_at < end)
                advance(a, next, NW);
        }
        cp_async_commit();
        return mk;
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i)
        masks[i] = request(i);

    typename StateOf<T, D, GP>::type st;
    int mine = at + warp;                                // this warp's next tile to attend
    int slot = 0;
    const int at0 = at;
    do {
        // the segment: tiles [at, seg_end) of unit (cur.b, cur.h), from its tile cur.s on
        const int left = SMALL ? end - at : cur.nt - cur.s;
        const int seg_end = at + left < end ? at + left : end;
        if constexpr (std::is_same<T, float>::value) {
            const float *qp = static_cast<const float *>(a.q) + (int64_t)cur.b * a.qs0 + (int64_t)cur.h * a.G * a.qs1;
            for (int i = threadIdx.x; i < GP * D; i += NW * 32)
                qs[i] = i / D < a.G ? qp[(int64_t)(i / D) * a.qs1 + i % D] : 0.f;
            __syncthreads();
        }
        const int unit = cur.b * a.Hkv + cur.h;
        st.begin(a, cur.b, cur.h, lane, qs);
        for (; mine < seg_end; mine += NW) {
            cp_async_wait<ST - 2>();
            __syncwarp();
            const int t0 = (cur.s + mine - at) * TT;
            float *lg = nullptr;
            if (SMALL && a.mass)
                lg = cm + 2 * kMaxG + (mine - at) * TT * a.G;
            else if (a.logits)
                lg = a.logits + ((int64_t)unit * a.max_tokens + t0) * a.G;
            unsigned mk = masks[0];
#pragma unroll
            for (int i = 0; i + 1 < ST; ++i)
                masks[i] = masks[i + 1];
            st.tile(a, ring + slot * S::tile_bytes, mk, cur.L - t0, lg, ps + warp * TT * GP, lane);
            __syncwarp();
            // Refill the slot freed a round ago.  Before the products instead,
            // the warps' requests bunch up: 169 against 163 us for 1.07 GB.
            masks[ST - 2] = request(slot == 0 ? ST - 1 : slot - 1);
            slot = slot + 1 == ST ? 0 : slot + 1;
        }
        st.end(a, ml + warp * 2 * kMaxG, po + warp * GP * D, lane);
        __syncthreads();
        if constexpr (SMALL) {
            join_cluster<T, D, GP>(a, cur, at0, end, C, rank, ml, po, cm, cm + 2 * kMaxG);
            break;
        }
        // join the warps' parts; a unit that lies wholly in this share is finished here
        const bool first = cur.s == 0, last = seg_end - at == left;
        float *part = a.parts + ((int64_t)cta * 2 + (first ? 1 : 0)) * part_floats(a.G, D);
        for (int i = threadIdx.x; i < a.G * D; i += NW * 32) {
            const int g = i / D, d = i - g * D;
            float mm = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < NW; ++w)
                mm = fmaxf(mm, ml[w * 2 * kMaxG + g]);
            const float base = or_zero(mm);
            float ll = 0.f, oo = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = weight(a, ml[w * 2 * kMaxG + g], base);
                ll = fmaf(f, ml[w * 2 * kMaxG + kMaxG + g], ll);
                oo = fmaf(f, po[(w * GP + g) * D + d], oo);
            }
            const int head = cur.h * a.G + g;
            if (first && last) {
                store_out(a, cur.b, head, d, ll > 0.f || ll != ll ? oo / ll : 0.f);
                if (d == 0) {
                    if (a.lse)
                        a.lse[(int64_t)cur.b * a.ls0 + (int64_t)head * a.ls1] = lse_of(a, mm, ll);
                    if (a.mass)
                        a.unit_sum[(int64_t)unit * a.G + g] = make_float2(mm, ll);
                }
            } else {
                if (d == 0) {
                    part[g] = mm;
                    part[kMaxG + g] = ll;
                }
                part[2 * kMaxG + i] = oo;
            }
        }
        __syncthreads();
        at = seg_end;
        if (at < end)
            advance(a, cur, left);
    } while (at < end);
    cp_async_wait<0>();
}

// Joins the parts of units that several CTAs shared (blockIdx.x < join_x, each
// join_heads heads of a unit), and with mass adds each token's weight, one CTA
// per (run of tokens, unit).  What a CTA reads goes out at once: the first
// parts, or a run's logits, before the heads' sums are known.  The parts'
// groups of threads are added in a fixed order.
constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 4;       // parts a thread requests first
constexpr int kMassTokens = 1024;   // tokens a CTA adds up

template <int D, int GP>
__global__ void __launch_bounds__(kJoinThreads, GP <= 4 ? 3 : 2) art_split_join_kernel(const __grid_constant__ SplitArgs a)
{
    constexpr int LPR = D / 4;                           // threads on one head's 16-byte columns
    __shared__ float4 sums[kJoinThreads];
    __shared__ float ms[kMaxG], ls[kMaxG];               // the heads' max and sum
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool weights = blockIdx.x >= a.join_x;
    const int g0 = weights ? 0 : blockIdx.x * a.join_heads, nh = weights ? a.G : min(a.join_heads, a.G - g0);
    const int t0 = ((int)blockIdx.x - a.join_x) * kMassTokens;
    // the lengths are inputs, complete before the first kernel started: the
    // shares are worked out while it still runs
    const Chunk chunk = chunk_of(a, 0, lane);
    const int total = batch_tiles(a, chunk, lane);
    const int n = sharers(a, total);
    bool waited = false;
    auto wait = [&] {
        if (!waited)
            follow();
        waited = true;
    };
    int before = 0;                                      // tiles of the sequences before b0, one kv-head
    int b0 = 0;
    Chunk here = chunk;
    for (int unit = blockIdx.y; unit < a.B * a.Hkv; unit += gridDim.y) {
        const int b = unit / a.Hkv, h = unit - b * a.Hkv;
        while (b >= b0 + 32) {
            before += (int)__shfl_sync(0xffffffffu, here.inc, 31);
            b0 += 32;
            here = chunk_of(a, b0, lane);
        }
        const int L = __shfl_sync(0xffffffffu, here.L, b - b0), nt = tiles_of(a, L);
        if (blockIdx.x == 0 && threadIdx.x == 0 && h == 0 && __ldcg(a.sl + b) > L)
            report(a.status, ART_ERR_BAD_INDEX);
        if (weights && t0 >= L)
            continue;
        if (nt == 0) {
            wait();
            for (int i = threadIdx.x; i < nh * D; i += kJoinThreads) {
                store_out(a, b, h * a.G + g0 + i / D, i % D, 0.f);
                if (i % D == 0 && a.lse)
                    a.lse[(int64_t)b * a.ls0 + (int64_t)(h * a.G + g0 + i / D) * a.ls1] = -CUDART_INF_F;
            }
            continue;
        }
        const int u0 = (before + (int)__shfl_sync(0xffffffffu, here.inc, b - b0) - nt) * a.Hkv + h * nt;
        const int c0 = share_of(u0, total, n), c1 = share_of(u0 + nt - 1, total, n);
        const bool joined = c1 > c0;
        if (!joined && !weights)
            continue;
        // part of CTA c: c0 met the unit's first tile (its slot 1), the others a later one (slot 0)
        const int pf = 2 * kMaxG + a.G * D;
        auto part = [&](int c) { return a.parts + (c * 2 + (c == c0 ? 1 : 0)) * pf; };
        // max and sum of the CTA's heads over the parts, a warp each, into ms and ls
        auto stats = [&] {
            if (warp < nh) {
                const int g = g0 + warp;
                float mm = -CUDART_INF_F, ll = 0.f;
                if (joined) {
                    for (int c = c0 + lane; c <= c1; c += 32) {
                        const float pm = part(c)[g], pl = part(c)[kMaxG + g];
                        const float top = fmaxf(mm, pm), base = or_zero(top);
                        ll = fmaf(ll, weight(a, mm, base), pl * weight(a, pm, base));
                        mm = top;
                    }
                    float top = mm;
#pragma unroll
                    for (int o = 16; o; o >>= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    ll *= weight(a, mm, or_zero(top));
#pragma unroll
                    for (int o = 16; o; o >>= 1)
                        ll += __shfl_xor_sync(0xffffffffu, ll, o);
                    mm = top;
                } else {
                    const float2 done = a.unit_sum[(int64_t)unit * a.G + g];
                    mm = done.x;
                    ll = done.y;
                }
                if (lane == 0) {
                    ms[warp] = mm;
                    ls[warp] = ll;
                }
            }
            __syncthreads();
        };
        if (!weights) {
            const int cols = nh * LPR;                   // 16-byte columns: 16 .. 512
            const int wide = cols < kJoinThreads ? cols : kJoinThreads, groups = kJoinThreads / wide;
            const int grp = threadIdx.x / wide;
            wait();
            for (int c4 = threadIdx.x % wide; c4 < cols; c4 += wide) {   // once but for wide heads
                const int g = c4 / LPR;
                const int col = 2 * kMaxG + g0 * D + c4 * 4;
                float4 x[kJoinAhead];
                float pm[kJoinAhead];
#pragma unroll
                for (int j = 0; j < kJoinAhead; ++j) {
                    const int c = c0 + grp + j * groups;
                    pm[j] = -CUDART_INF_F;
                    x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (c <= c1 && grp < groups) {
                        pm[j] = part(c)[g0 + g];
                        x[j] = *reinterpret_cast<const float4 *>(part(c) + col);
                    }
                }
                if (c4 < wide)
                    stats();
                const float base = or_zero(ms[g]);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                auto add = [&](float m, const float4 &v) {
                    const float f = weight(a, m, base);
                    o.x = fmaf(f, v.x, o.x);
                    o.y = fmaf(f, v.y, o.y);
                    o.z = fmaf(f, v.z, o.z);
                    o.w = fmaf(f, v.w, o.w);
                };
#pragma unroll
                for (int j = 0; j < kJoinAhead; ++j)
                    add(pm[j], x[j]);
                if (grp < groups)
                    for (int c = c0 + grp + kJoinAhead * groups; c <= c1; c += groups)
                        add(part(c)[g0 + g], *reinterpret_cast<const float4 *>(part(c) + col));
                if (groups > 1) {
                    sums[threadIdx.x] = o;
                    __syncthreads();
                    for (int i = 1; grp == 0 && i < groups; ++i) {
                        const float4 y = sums[i * wide + c4];
                        o.x += y.x;
                        o.y += y.y;
                        o.z += y.z;
                        o.w += y.w;
                    }
                }
                if (grp == 0) {
                    const bool some = ls[g] > 0.f || ls[g] != ls[g];
                    const float *ov = &o.x;
                    const int head = h * a.G + g0 + g, d = (c4 % LPR) * 4;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        store_out(a, b, head, d + e, some ? ov[e] / ls[g] : 0.f);
                    if (d == 0 && a.lse)
                        a.lse[(int64_t)b * a.ls0 + (int64_t)head * a.ls1] = lse_of(a, ms[g], ls[g]);
                }
            }
        } else {
            // tokens left out of the attention have a logit of -inf: they gain 0
            constexpr int N = kMassTokens / kJoinThreads;
            const float *lg = a.logits + unit * a.max_tokens * a.G + (int64_t)t0 * a.G;
            float *mrow = a.mass + (int64_t)b * a.ms0 + (int64_t)h * a.ms1 + t0;
            const int left = L - t0;
            float old[N], x[N][GP];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int t = threadIdx.x + i * kJoinThreads;
                old[i] = t < left ? __ldcg(mrow + t) : 0.f;
            }
            wait();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int t = threadIdx.x + i * kJoinThreads;
                if (t < left && a.G % 4 == 0) {
#pragma unroll
                    for (int g = 0; g < GP; g += 4)
                        if (g < a.G)
                            *reinterpret_cast<float4 *>(&x[i][g]) = *reinterpret_cast<const float4 *>(lg + t * a.G + g);
                } else if (t < left) {
#pragma unroll
                    for (int g = 0; g < GP; ++g)
                        if (g < a.G)
                            x[i][g] = lg[t * a.G + g];
                }
            }
            stats();
            if (threadIdx.x < a.G) {
                ms[threadIdx.x] = or_zero(ms[threadIdx.x]);
                ls[threadIdx.x] = ls[threadIdx.x] == 0.f ? 0.f : log2f(ls[threadIdx.x]);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int t = threadIdx.x + i * kJoinThreads;
                if (t < left) {
                    float w = 0.f;
#pragma unroll
                    for (int g = 0; g < GP; ++g)
                        if (g < a.G)
                            w += ex2_approx(fmaf(x[i][g] - ms[g], a.scale_log2, -ls[g]));
                    mrow[t] = old[i] + w;
                }
            }
        }
        __syncthreads();                                 // sums, ms, ls are rewritten for the next unit
    }
    wait();
}

// --------------------------------------------------------------- host ----

struct Plan {
    int G, D, bf16, ctas, least, tile_log, cluster;
    int64_t units, max_tokens, parts_bytes, sums_bytes, logits_bytes;
    int64_t bytes() const { return parts_bytes + sums_bytes + logits_bytes; }
};

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

bool has(const art_tensor_t &t) { return t.data != nullptr; }

// out: whether the call writes one (the workspace query needs none)
art_status_t plan_of(const art_split_params_t *p, bool out, Plan *pl)
{
    const art_tensor_t *q = &p->q, *k = &p->k_cache, *v = &p->v_cache, *pt = &p->page_table, *sl = &p->seq_lens,
                       *o = &p->out;
    if (is_null(q) || is_null(k) || is_null(v) || is_null(pt) || is_null(sl) || (out && is_null(o)))
        return ART_ERR_NULL;
    if (q->ndim != 3 || k->ndim != 4 || v->ndim != 4 || pt->ndim != 2 || sl->ndim != 1 || (out && o->ndim != 3) ||
        (has(p->lse) && p->lse.ndim != 2) || (has(p->mass) && p->mass.ndim != 3))
        return ART_ERR_SHAPE;
    if ((q->dtype != ART_F32 && q->dtype != ART_BF16) || k->dtype != q->dtype || v->dtype != q->dtype ||
        pt->dtype != ART_I32 || sl->dtype != ART_I32 || (out && o->dtype != ART_F32 && o->dtype != ART_BF16) ||
        (has(p->lse) && p->lse.dtype != ART_F32) || (has(p->mass) && p->mass.dtype != ART_F32))
        return ART_ERR_DTYPE;
    const int64_t B = q->shape[0], Hq = q->shape[1], d = q->shape[2];
    const int64_t NP = k->shape[0], Hkv = k->shape[1], page = k->shape[2], mb = pt->shape[1];
    if (B <= 0 || Hq <= 0 || d <= 0 || NP <= 0 || Hkv <= 0 || page <= 0 || mb <= 0 || B > 65535 || Hq > 4096 ||
        NP > (int64_t)INT32_MAX || page > 4096 || mb * page > (int64_t)INT32_MAX - 4096)
        return ART_ERR_SHAPE;
    for (int i = 0; i < 4; ++i)
        if (v->shape[i] != k->shape[i])
            return ART_ERR_SHAPE;
    if (k->shape[3] != d || Hq % Hkv || pt->shape[0] != B || sl->shape[0] != B ||
        (out && (o->shape[0] != B || o->shape[1] != Hq || o->shape[2] != d)))
        return ART_ERR_SHAPE;
    if (has(p->lse) && (p->lse.shape[0] != B || p->lse.shape[1] != Hq))
        return ART_ERR_SHAPE;
    if (has(p->mass) && (p->mass.shape[0] != B || p->mass.shape[1] != Hkv || p->mass.shape[2] < mb * page))
        return ART_ERR_SHAPE;
    const int64_t es = elem_size(q->dtype);
    if (q->stride[2] != 1 || k->stride[3] != 1 || v->stride[3] != 1 || pt->stride[1] != 1 || sl->stride[0] != 1 ||
        (out && o->stride[2] != 1) || pt->stride[0] < 0)
        return ART_ERR_SHAPE;
    if (!aligned(q->data, 16) || (q->stride[0] * es) % 16 || (q->stride[1] * es) % 16 || q->stride[0] < 0 ||
        q->stride[1] < 0)
        return ART_ERR_SHAPE;
    for (const art_tensor_t *c : {k, v}) {
        if (!aligned(c->data, 16))
            return ART_ERR_SHAPE;
        for (int i = 0; i < 3; ++i)
            if (c->stride[i] <= 0 || (c->stride[i] * es) % 16)
                return ART_ERR_SHAPE;
    }
    // written tensors: elements may not overlap
    if (out && (!apart(*o) || !aligned(o->data, elem_size(o->dtype))))
        return ART_ERR_SHAPE;
    if (has(p->lse) && (!aligned(p->lse.data, 4) || !apart(p->lse)))
        return ART_ERR_SHAPE;
    if (has(p->mass) && (!aligned(p->mass.data, 4) || p->mass.stride[2] != 1 || !apart(p->mass)))
        return ART_ERR_SHAPE;
    if (!aligned(pt->data, 4) || !aligned(sl->data, 4) || (p->device_status && !aligned(p->device_status, 4)))
        return ART_ERR_SHAPE;
    // the products are scaled to base 2 in one step, which has to be a number too
    if (!std::isfinite(p->sm_scale) || !std::isfinite((float)(p->sm_scale * kLog2e)))
        return ART_ERR_PARAM;
    const int64_t G = Hq / Hkv;
    if (!(d == 64 || d == 128 || d == 256) || G > kMaxG)
        return ART_ERR_UNSUPPORTED;
    pl->G = (int)G;
    pl->D = (int)d;
    pl->bf16 = q->dtype == ART_BF16;
    pl->units = B * Hkv;
    pl->max_tokens = mb * page;
    pl->tile_log = !pl->bf16 && (d == 256 || (d == 128 && G <= 4)) ? 3 : 4;   // kTileOf's and Shape's rules
    const int64_t rows = 1 << pl->tile_log;
    const bool big = 2 * rows * d * es > 8192;
    pl->ctas = art_stream::sm_count() * (big ? 1 : 2);
    pl->least = (int)((big ? 128 : 64) / rows);
    // Short units, and few of them: one kernel, with a cluster of CTAs on each
    // unit (at most 128 tokens a CTA, or 64), instead of two.  Measured: 8 units
    // of 1024 tokens 5.7 us, shared out evenly 6.9; 64 of 512 7.5 and 10.0; 512
    // of 100 12.2 and 16.0; but 64 units of 1024 13.8 and 12.8.
    const int64_t tiles = (pl->max_tokens + rows - 1) / rows, most = rows == 8 ? 16 : pl->bf16 && d == 256 && G > 4 ? 4 : 8;
    if (pl->units * tiles > (int64_t)INT32_MAX)
        return ART_ERR_UNSUPPORTED;
    pl->cluster = 1;
    while (pl->cluster < kMaxCluster && pl->cluster * most < tiles)
        pl->cluster *= 2;
    if (pl->cluster * most < tiles || pl->units * tiles * rows > 65536 || (pl->cluster > 1 && pl->units * pl->cluster > pl->ctas))
        pl->cluster = 0;
    if (pl->cluster) {
        pl->parts_bytes = pl->sums_bytes = pl->logits_bytes = 0;
        return ART_OK;
    }
    pl->parts_bytes = up256((int64_t)pl->ctas * 2 * part_floats(G, d) * 4);
    pl->sums_bytes = has(p->mass) ? up256(pl->units * G * 8) : 0;
    pl->logits_bytes = has(p->mass) ? up256(pl->units * G * pl->max_tokens * 4) : 0;
    return ART_OK;
}

template <typename T, int D, int GP>
cudaError_t launch_split(const SplitArgs &a, cudaStream_t s)
{
    using S = Shape<T, D, GP>;
    const int smem = a.cluster ? S::smem_cluster : S::smem;
    const auto fn = a.cluster ? art_split_kernel<T, D, GP, true> : art_split_kernel<T, D, GP, false>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    const int64_t units = (int64_t)a.B * a.Hkv;
    if (a.cluster)
        return art_stream::launch(fn, dim3((unsigned)(units * a.cluster)), S::warps * 32, smem, s, a, a.cluster);
    if ((e = art_stream::launch(fn, dim3((unsigned)a.ctas), S::warps * 32, smem, s, a)) != cudaSuccess)
        return e;
    const int64_t runs = a.mass ? (a.max_tokens + kMassTokens - 1) / kMassTokens : 0;
    return art_stream::launch(art_split_join_kernel<D, GP>,
                              dim3((unsigned)(a.join_x + runs), (unsigned)(units < 65535 ? units : 65535)), kJoinThreads, 0, s, a);
}

template <typename T, int D>
cudaError_t launch_split_g(const SplitArgs &a, cudaStream_t s)
{
    return a.G <= 4 ? launch_split<T, D, 4>(a, s) : launch_split<T, D, 8>(a, s);
}

template <typename T>
cudaError_t launch_split_d(const SplitArgs &a, int d, cudaStream_t s)
{
    return d == 64 ? launch_split_g<T, 64>(a, s) : d == 128 ? launch_split_g<T, 128>(a, s) : launch_split_g<T, 256>(a, s);
}

}  // namespace

extern "C" {

int64_t art_split_workspace_bytes(const art_split_params_t *p)
{
    if (!p)
        return ART_ERR_NULL;
    Plan pl;
    const art_status_t st = plan_of(p, has(p->out), &pl);
    return st == ART_OK ? pl.bytes() : (int64_t)st;
}

art_status_t art_decode_attention_split(const art_split_params_t *p, art_stream_t stream)
{
    if (!p)
        return ART_ERR_NULL;
    Plan pl;
    const art_status_t st = plan_of(p, true, &pl);
    if (st != ART_OK)
        return st;
    if (p->out.data == p->q.data)
        return ART_ERR_PARAM;
    if (pl.bytes() > 0 && !p->workspace)
        return ART_ERR_NULL;
    if (p->workspace_bytes < pl.bytes() || !aligned(p->workspace, 256))
        return ART_ERR_SHAPE;
    SplitArgs a;
    const int64_t es = elem_size(p->q.dtype);
    a.q = p->q.data;
    a.qs0 = p->q.stride[0];
    a.qs1 = p->q.stride[1];
    a.k = p->k_cache.data;
    a.ks0 = p->k_cache.stride[0] * es;
    a.ks1 = p->k_cache.stride[1] * es;
    a.ks2 = p->k_cache.stride[2] * es;
    a.v = p->v_cache.data;
    a.vs0 = p->v_cache.stride[0] * es;
    a.vs1 = p->v_cache.stride[1] * es;
    a.vs2 = p->v_cache.stride[2] * es;
    a.pt = static_cast<const int32_t *>(p->page_table.data);
    a.pts0 = p->page_table.stride[0];
    a.sl = static_cast<const int32_t *>(p->seq_lens.data);
    a.out = p->out.data;
    a.os0 = p->out.stride[0];
    a.os1 = p->out.stride[1];
    a.out_bf16 = p->out.dtype == ART_BF16;
    a.lse = static_cast<float *>(p->lse.data);
    a.ls0 = p->lse.stride[0];
    a.ls1 = p->lse.stride[1];
    a.mass = static_cast<float *>(p->mass.data);
    a.ms0 = p->mass.stride[0];
    a.ms1 = p->mass.stride[1];
    a.B = (int)p->q.shape[0];
    a.Hq = (int)p->q.shape[1];
    a.Hkv = (int)p->k_cache.shape[1];
    a.G = pl.G;
    a.page = (int)p->k_cache.shape[2];
    a.max_blocks = (int)p->page_table.shape[1];
    a.num_pages = (int)p->k_cache.shape[0];
    a.tile_log = pl.tile_log;
    a.page_whole = a.page % (1 << pl.tile_log) == 0;
    a.scale_log2 = (float)((p->sm_scale > 0.f ? (double)p->sm_scale : 1.0 / std::sqrt((double)pl.D)) * kLog2e);
    a.status = p->device_status;
    a.ctas = pl.ctas;
    a.cluster = pl.cluster;
    // few units have many parts each: a CTA a head; many units: a CTA each
    a.join_heads = pl.units >= 128 ? pl.G : 1;
    a.join_x = (pl.G + a.join_heads - 1) / a.join_heads;
    a.least = pl.least;
    uint8_t *ws = static_cast<uint8_t *>(p->workspace);
    a.parts = reinterpret_cast<float *>(ws);
    a.unit_sum = pl.sums_bytes ? reinterpret_cast<float2 *>(ws + pl.parts_bytes) : nullptr;
    a.logits = pl.logits_bytes ? reinterpret_cast<float *>(ws + pl.parts_bytes + pl.sums_bytes) : nullptr;
    a.max_tokens = pl.max_tokens;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = pl.bf16 ? launch_split_d<__nv_bfloat16>(a, pl.D, s) : launch_split_d<float>(a, pl.D, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return ART_ERR_LAUNCH;
    }
    return ART_OK;
}

}  // extern "C"
