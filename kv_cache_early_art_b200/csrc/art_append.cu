// art_append.cu -- rotary positions on new tokens' queries and keys, and their
// keys and values written into the paged cache (art_rope_init,
// art_rope_init_freqs, art_rope_append in art.h).
//
// Channel pair i of a head at position p turns by the angle p f_i:
//     (x, y) -> a (x cos - y sin, x sin + y cos),
// a the amplitude.  Far positions are what costs precision: p f_i in 32 bits is
// off by up to 2^-24 of the angle, 0.01 rad at p = 10^5.  Here f_i is held as
// the 64-bit fraction of a turn a position adds, F_i = 2^64 frac(f_i / 2 pi)
// to the nearest whole number; p F_i modulo 2^64 is then the fraction of the
// angle's last turn, to 2^-34 of a turn for any 32-bit position and at the price
// of one integer product.  Its leading 32 bits enter the sines whole (turn()).
//
// Bound by memory: every element is read once and written once (489 MB, 24.5k
// tokens of 28 + 2 * 4 heads of 128: 78 us, 96 % of the measured copy rate).  A
// thread owns two 16-byte vectors of a head (E whole pairs in either layout) for one token, so it turns its angles into sines once
// and uses them for all the heads it walks.  With few tokens the heads of a
// token are spread over many threads instead (latency: 3.6 us for eight
// tokens), with many tokens over few.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "../../include/art.h"
#include "art_host.h"
#include "art_stream.cuh"

namespace {

using art_host::aligned;
using art_host::apart;
using art_host::elem_size;
using art_host::is_null;

constexpr int kThreads = 256;
constexpr int kAhead = 4;       // heads a thread has in flight
constexpr int kRing = kAhead * 2 * kThreads * 16;
static_assert(kRing <= 48 * 1024, "no opt-in to larger shared memory");

struct AppendArgs {
    const void *q, *k, *v;
    void *qo, *kc, *vc;
    int64_t qs0, qs1, ks0, ks1, vs0, vs1, qos0, qos1;   // token, head strides (elements)
    int64_t kc0, kc1, kc2, vc0, vc1, vc2;               // page, head, token strides
    const int32_t *pt;
    int64_t pts0;
    const int32_t *slots, *pos, *seq;
    float *mass;
    int64_t ms0, ms1;
    int T, B, Hq, Hkv, d, page, max_blocks, num_pages;
    int units;          // threads on a head: two vectors each (row kernel: one; scalar: pairs and single channels)
    int lanes;          // threads (row kernel: warps) that share the heads of one (token, unit)
    int group;          // row kernel: lanes on a head's row
    int32_t *status;
    art_rope_t rope;
};

__device__ __forceinline__ void report(int32_t *status, int32_t code)
{
    if (status)
        atomicCAS(status, 0, code);
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int E = 4;
    __device__ static __forceinline__ void unpack(const uint4 &v, float *f)
    {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    __device__ static __forceinline__ uint4 pack(const float *f)
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    __device__ static __forceinline__ float get(const float *p) { return *p; }
    __device__ static __forceinline__ void put(float *p, float v) { *p = v; }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int E = 8;
    __device__ static __forceinline__ void unpack(const uint4 &v, float *f)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static __forceinline__ uint4 pack(const float *f)
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    __device__ static __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
};

// Cosine and sine (times the amplitude) of pair i at a position.  The angle's
// leading 32 bits are taken to the nearest quarter turn in integers; the rest, an
// eighth of a turn at most, becomes x + y radians (x the float nearest to most of
// it), and the sines are Taylor's polynomials in x, turned on by y to first
// order: remainders x^11 / 11! and x^12 / 12! below 2^-29 and 2^-33 at pi / 4, y
// below 2^-23, roundings 1.5 steps of the result at most.  So the angle is right
// to 2^-32 of a turn; the fraction handed to sincospif as one float was off by up
// to 2^-26, the sines by 1.1e-7, in the same time (24k tokens of 28 + 2 * 4 heads
// of 128 69.6 us; sincospif and a correction of its results 69.8).
__device__ __forceinline__ void turn(const art_rope_t &r, int i, int32_t pos, float &c, float &s)
{
    constexpr double kUnit = 6.283185307179586476925286766559 * 0x1p-32;        // radians
    constexpr float kHigh = (float)kUnit, kLow = (float)(kUnit - (double)kHigh);
    const uint64_t frac = r.turns[i] * (uint64_t)(int64_t)pos;      // of a turn, modulo 1
    const uint32_t top = (uint32_t)((frac + 0x80000000u) >> 32);
    const uint32_t quarter = (top + (1u << 29)) >> 30;              // the nearest, modulo 4
    const int32_t rest = (int32_t)(top - (quarter << 30));
    const float lead = (float)rest;
    const float x = lead * kHigh, x2 = x * x;
    const float y = fmaf((float)(rest - (int32_t)lead), kHigh, fmaf(lead, kLow, fmaf(lead, kHigh, -x)));
    float p = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f), q = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
    p = fmaf(x2, p, 1.f / 120.f);
    q = fmaf(x2, q, -1.f / 720.f);
    p = fmaf(x2, p, -1.f / 6.f) * x2;
    q = fmaf(x2, q, 1.f / 24.f);
    const float c0 = fmaf(x2, fmaf(x2, q, -0.5f), 1.f);
    const float s1 = x + fmaf(x, p, c0 * y), c1 = fmaf(-x, y, c0);  // (x for sin x: below 2^-26 apart)
    c = (quarter & 1) ? -s1 : c1;
    s = (quarter & 1) ? c1 : s1;
    const float a = (quarter & 2) ? -r.amplitude : r.amplitude;
    c *= a;
    s *= a;
}

// where a token goes: looked up, and (settle) judged later
struct Spot {
    int seq, slot, pos, pg;      // pg: -1 out of range, -2 padding
};
__device__ __forceinline__ Spot find_spot(const AppendArgs &a, int t)
{
    Spot p;
    p.seq = a.seq ? a.seq[t] : t;
    p.slot = a.slots[t];
    p.pos = a.pos ? a.pos[t] : p.slot;
    p.pg = -2;
    if (p.seq >= 0 && p.slot >= 0) {
        p.pg = -1;
        if (p.seq < a.B && p.slot / a.page < a.max_blocks)
            p.pg = a.pt[(int64_t)p.seq * a.pts0 + p.slot / a.page];
        if (p.pg < 0 || p.pg >= a.num_pages)
            p.pg = -1;
    }
    return p;
}
__device__ __forceinline__ bool settle(const AppendArgs &a, const Spot &p, bool tell)
{
    if (p.pg == -1 && tell)
        report(a.status, ART_ERR_BAD_INDEX);
    return p.pg >= 0;
}

// a vector of channels e0 ..: the new value below rot (even), untouched behind it
template <typename T>
__device__ __forceinline__ uint4 turned(const uint4 &old, const uint4 &now, int e0, int rot)
{
    constexpr int W = Vec<T>::E / 4;
    return make_uint4(e0 < rot ? now.x : old.x, e0 + W < rot ? now.y : old.y, e0 + 2 * W < rot ? now.z : old.z,
                      e0 + 3 * W < rot ? now.w : old.w);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Heads are numbered q 0 .. Hq-1, then k, then v.  A thread walks its heads of
// one token and keeps kAhead of them in flight in shared memory, by
// asynchronous copies into places of its own that it alone reads: no barrier
// anywhere, and the look-ups and the sines hide behind the first ones.  (489
// MB: 78 us; 93 us with the loads in registers, which held two to four heads; 90 us
// with resident CTAs that went on to further tokens, whose look-ups did not
// hide.)
template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kThreads, 3) art_append_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr int E = Vec<T>::E;
    extern __shared__ __align__(128) uint4 ring[];       // [kAhead][2][kThreads]
    art_stream::follow();
    const int per = a.units * a.lanes, tpb = kThreads / per;
    const int tib = threadIdx.x / per;
    const int in = threadIdx.x - tib * per;
    const int t = blockIdx.x * tpb + tib;
    const int hl = in / a.units, u = in - hl * a.units;
    const int nqk = a.Hq + a.Hkv, nh = nqk + a.Hkv;
    if (tib >= tpb || t >= a.T || hl >= nh)
        return;
    const int rot = a.rope.rot_dim;
    // The thread's two vectors: the u-th of the head's first and second half, so
    // that neighbouring threads read neighbouring vectors (453 MB interleaved, 64 of
    // 128 turning: 71 us; 106 us with 32 adjacent bytes a thread).  ART_ROPE_HALF (rot
    // a multiple of 2 E) halves the turning channels so, and those behind them.
    const int w0 = u * E, w1 = a.d / 2 + u * E;
    int o0 = w0, o1 = w1, turning = a.units;
    if (LAYOUT == ART_ROPE_HALF) {
        turning = rot / (2 * E);
        if (u < turning) {
            o1 = rot / 2 + u * E;
        } else {
            o0 = rot / 2 + u * E;
            o1 = o0 + (a.d - rot) / 2;
        }
    }
    const T *qp = static_cast<const T *>(a.q) + (int64_t)t * a.qs0;
    const T *kp = static_cast<const T *>(a.k) + (int64_t)t * a.ks0;
    const T *vp = static_cast<const T *>(a.v) + (int64_t)t * a.vs0;
    const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring + threadIdx.x);
    int fh = hl, fslot = 0;                              // the head to request next
    auto request = [&] {
        if (fh < nh) {
            const bool v = fh >= nqk;
            const T *src = fh < a.Hq ? qp + (int64_t)fh * a.qs1
                                     : v ? vp + (int64_t)(fh - nqk) * a.vs1 : kp + (int64_t)(fh - a.Hq) * a.ks1;
            const uint32_t dst = mine + fslot * (2 * kThreads * 16);
            cp_async16(dst, src + (v ? w0 : o0));
            cp_async16(dst + kThreads * 16, src + (v ? w1 : o1));
            fh += a.lanes;
        }
        fslot = fslot + 1 == kAhead ? 0 : fslot + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i)
        request();
    const Spot here = find_spot(a, t);
    if (settle(a, here, in == 0)) {
        const int64_t row = here.slot % a.page;
        if (a.mass && u == 0)
            for (int h = hl; h < a.Hkv; h += a.lanes)
                a.mass[(int64_t)here.seq * a.ms0 + (int64_t)h * a.ms1 + here.slot] = 0.f;
        float c[E], s[E];
        if (u < turning && hl < nqk) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (LAYOUT == ART_ROPE_HALF) {
                    turn(a.rope, u * E + e, here.pos, c[e], s[e]);
                } else {
                    const int i = (e < E / 2 ? o0 / 2 : (o1 - E) / 2) + e;
                    c[e] = s[e] = 0.f;
                    if (2 * i < rot)
                        turn(a.rope, i, here.pos, c[e], s[e]);
                }
            }
        }
        T *qo = static_cast<T *>(a.qo) + (int64_t)t * a.qos0;
        T *ko = static_cast<T *>(a.kc) + (int64_t)here.pg * a.kc0 + row * a.kc2;
        T *vo = static_cast<T *>(a.vc) + (int64_t)here.pg * a.vc0 + row * a.vc2;
        int slot = 0;
        for (int h = hl; h < nh; h += a.lanes) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
            uint4 x = ring[slot * 2 * kThreads + threadIdx.x], y = ring[(slot * 2 + 1) * kThreads + threadIdx.x];
            request();                                   // into the place read a head ago
            slot = slot + 1 == kAhead ? 0 : slot + 1;
            const bool v = h >= nqk;
            if (u < turning && !v) {
                float f[2 * E], g[2 * E];
                Vec<T>::unpack(x, f);
                Vec<T>::unpack(y, f + E);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i0 = LAYOUT == ART_ROPE_HALF ? e : 2 * e, i1 = LAYOUT == ART_ROPE_HALF ? E + e : 2 * e + 1;
                    g[i0] = fmaf(f[i0], c[e], -(f[i1] * s[e]));
                    g[i1] = fmaf(f[i0], s[e], f[i1] * c[e]);
                }
                if (LAYOUT == ART_ROPE_HALF) {
                    x = Vec<T>::pack(g);
                    y = Vec<T>::pack(g + E);
                } else {
                    x = turned<T>(x, Vec<T>::pack(g), o0, rot);
                    y = turned<T>(y, Vec<T>::pack(g + E), o1, rot);
                }
            }
            T *dst = h < a.Hq ? qo + (int64_t)h * a.qos1
                              : v ? vo + (int64_t)(h - nqk) * a.vc1 : ko + (int64_t)(h - a.Hq) * a.kc1;
            *reinterpret_cast<uint4 *>(dst + (v ? w0 : o0)) = x;
            *reinterpret_cast<uint4 *>(dst + (v ? w1 : o1)) = y;
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ART_ROPE_HALF where half of rot_dim is no whole number of vectors: a pair's
// channels then sit at different places of their vectors.  A group of lanes
// takes a head's row, one 16-byte vector each (two each for 256 fp32 channels),
// from the same kind of ring, and reads the partners of its channels from its
// neighbours' places there.  (453 MB at 100 of 128 turning: 94 us, 74 % of the
// measured copy rate; 266 us by the kernel below, pair by pair.  What is left is
// instructions: at six of 128 turning it takes as long.  Rings of six or eight
// rows and hoisted partner places gave nothing or cost a resident CTA.)
template <typename T>
__global__ void __launch_bounds__(kThreads) art_append_row_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr int E = Vec<T>::E, W = E / 4;              // channels of a vector, of a 32-bit word
    constexpr int NV = sizeof(T) == 4 ? 2 : 1;           // vectors a lane may have
    __shared__ uint4 ring[kThreads / 32][kAhead][32 * NV];
    __shared__ float2 sines[kThreads / 32][ART_ROPE_MAX_PAIRS];
    art_stream::follow();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + warp;
    const int t = (int)(item / a.lanes), share = (int)(item - (int64_t)t * a.lanes);
    if (t >= a.T)
        return;                                          // the whole warp
    const int nqk = a.Hq + a.Hkv, nh = nqk + a.Hkv;
    const int sl = lane % a.group, gi = lane / a.group, per = 32 / a.group;
    const T *qp = static_cast<const T *>(a.q) + (int64_t)t * a.qs0;
    const T *kp = static_cast<const T *>(a.k) + (int64_t)t * a.ks0;
    const T *vp = static_cast<const T *>(a.v) + (int64_t)t * a.vs0;
    // the group's row of a slot: units <= group, or group is the warp and units <= 32 NV
    const int base = gi * a.units, step = a.lanes * per;
    int fh = share * per + gi, fslot = 0;
    auto request = [&] {
        if (fh < nh) {
            const T *src = fh < a.Hq ? qp + (int64_t)fh * a.qs1
                                     : fh < nqk ? kp + (int64_t)(fh - a.Hq) * a.ks1 : vp + (int64_t)(fh - nqk) * a.vs1;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (sl + 32 * j < a.units)
                    cp_async16((uint32_t)__cvta_generic_to_shared(&ring[warp][fslot][base + sl + 32 * j]),
                               src + (sl + 32 * j) * E);
            fh += step;
        }
        fslot = fslot + 1 == kAhead ? 0 : fslot + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i)
        request();
    const Spot here = find_spot(a, t);
    if (settle(a, here, lane == 0 && share == 0)) {      // the same for the whole warp
        const int64_t row = here.slot % a.page;
        if (a.mass && share == 0)
            for (int h = lane; h < a.Hkv; h += 32)
                a.mass[(int64_t)here.seq * a.ms0 + (int64_t)h * a.ms1 + here.slot] = 0.f;
        const int rot = a.rope.rot_dim, hh = rot / 2;
        for (int i = lane; i < hh; i += 32) {
            float2 cs;
            turn(a.rope, i, here.pos, cs.x, cs.y);
            sines[warp][i] = cs;
        }
        __syncwarp();
        float c[NV][E], s[NV][E];                        // s: minus the sine for a pair's first channel
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int e = (sl + 32 * j) * E + i;
                const float2 cs = e < rot ? sines[warp][e < hh ? e : e - hh] : make_float2(0.f, 0.f);
                c[j][i] = cs.x;
                s[j][i] = e < hh ? -cs.y : cs.y;
            }
        T *qo = static_cast<T *>(a.qo) + (int64_t)t * a.qos0;
        T *ko = static_cast<T *>(a.kc) + (int64_t)here.pg * a.kc0 + row * a.kc2;
        T *vo = static_cast<T *>(a.vc) + (int64_t)here.pg * a.vc0 + row * a.vc2;
        int slot = 0;
        for (int h0 = share * per; h0 < nh; h0 += step) {
            const int h = h0 + gi;
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
            __syncwarp();                                // every lane's copies are in, and the last head's place is read
            request();
            const uint4 *mine = &ring[warp][slot][base];
            slot = slot + 1 == kAhead ? 0 : slot + 1;
            if (h < nh) {
                const T *from = reinterpret_cast<const T *>(mine);
                T *dst = h < a.Hq ? qo + (int64_t)h * a.qos1
                                  : h < nqk ? ko + (int64_t)(h - a.Hq) * a.kc1 : vo + (int64_t)(h - nqk) * a.vc1;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int e0 = (sl + 32 * j) * E;
                    if (sl + 32 * j >= a.units)
                        continue;
                    uint4 x = mine[sl + 32 * j];
                    if (h < nqk && e0 < rot) {
                        float f[E], y[E], g[E];
                        Vec<T>::unpack(x, f);
                        if (hh % W == 0) {               // partners in whole words
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int e = e0 + i * W;
                                w[i] = e < rot ? *reinterpret_cast<const uint32_t *>(from + (e < hh ? e + hh : e - hh)) : 0;
                            }
                            Vec<T>::unpack(make_uint4(w[0], w[1], w[2], w[3]), y);
                        } else {
#pragma unroll
                            for (int i = 0; i < E; ++i) {
                                const int e = e0 + i;
                                y[i] = e < rot ? Vec<T>::get(from + (e < hh ? e + hh : e - hh)) : 0.f;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < E; ++i)
                            g[i] = fmaf(f[i], c[j][i], y[i] * s[j][i]);
                        x = turned<T>(x, Vec<T>::pack(g), e0, rot);
                    }
                    *reinterpret_cast<uint4 *>(dst + e0) = x;
                }
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Any even rot_dim and any alignment: a thread takes a pair (units 0 ..
// rot / 2 - 1) or one channel behind them; for v, two neighbouring channels.
template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kThreads) art_append_scalar_kernel(const __grid_constant__ AppendArgs a)
{
    art_stream::follow();
    const int64_t n = (int64_t)a.T * a.units * a.lanes;
    for (int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x; it < n; it += (int64_t)gridDim.x * kThreads) {
        const int u = (int)(it % a.units);
        const int64_t r = it / a.units;
        const int hl = (int)(r % a.lanes), t = (int)(r / a.lanes);
        const Spot here = find_spot(a, t);
        if (!settle(a, here, u == 0 && hl == 0))
            continue;
        const int64_t row = here.slot % a.page;
        if (a.mass && u == 0)
            for (int h = hl; h < a.Hkv; h += a.lanes)
                a.mass[(int64_t)here.seq * a.ms0 + (int64_t)h * a.ms1 + here.slot] = 0.f;
        const int rot = a.rope.rot_dim;
        const bool pair = u < rot / 2;
        int i0 = rot + (u - rot / 2), i1 = i0;
        float c = 1.f, s = 0.f;
        if (pair) {
            i0 = LAYOUT == ART_ROPE_HALF ? u : 2 * u;
            i1 = LAYOUT == ART_ROPE_HALF ? u + rot / 2 : 2 * u + 1;
            turn(a.rope, u, here.pos, c, s);
        }
        const T *qp = static_cast<const T *>(a.q) + (int64_t)t * a.qs0;
        const T *kp = static_cast<const T *>(a.k) + (int64_t)t * a.ks0;
        const T *vp = static_cast<const T *>(a.v) + (int64_t)t * a.vs0;
        T *qo = static_cast<T *>(a.qo) + (int64_t)t * a.qos0;
        T *ko = static_cast<T *>(a.kc) + (int64_t)here.pg * a.kc0 + row * a.kc2;
        T *vo = static_cast<T *>(a.vc) + (int64_t)here.pg * a.vc0 + row * a.vc2;
        for (int h = hl; h < a.Hq + a.Hkv; h += a.lanes) {
            const T *src = h < a.Hq ? qp + (int64_t)h * a.qs1 : kp + (int64_t)(h - a.Hq) * a.ks1;
            T *dst = h < a.Hq ? qo + (int64_t)h * a.qos1 : ko + (int64_t)(h - a.Hq) * a.kc1;
            if (pair) {
                const float x = Vec<T>::get(src + i0), y = Vec<T>::get(src + i1);
                Vec<T>::put(dst + i0, fmaf(x, c, -(y * s)));
                Vec<T>::put(dst + i1, fmaf(x, s, y * c));
            } else {
                dst[i0] = src[i0];
            }
        }
        for (int h = hl; h < a.Hkv; h += a.lanes)
            for (int i = u; i < a.d; i += a.units)
                vo[(int64_t)h * a.vc1 + i] = vp[(int64_t)h * a.vs1 + i];
    }
}

// --------------------------------------------------------------- host ----

bool has(const art_tensor_t &t) { return t.data != nullptr; }

bool head_size(int64_t d) { return d > 0 && d % 16 == 0 && d <= 2 * ART_ROPE_MAX_PAIRS; }

bool vector_rows(const art_tensor_t &t, int nd)
{
    const int64_t es = elem_size(t.dtype);
    if (!aligned(t.data, 16))
        return false;
    for (int i = 0; i < nd - 1; ++i)
        if ((t.stride[i] * es) % 16)
            return false;
    return true;
}

enum Way { kPieces, kRows, kScalar };

template <typename T, int LAYOUT>
cudaError_t launch_layout(const AppendArgs &a, Way way, int grid, cudaStream_t s)
{
    return way == kPieces ? art_stream::launch(art_append_kernel<T, LAYOUT>, dim3((unsigned)grid), kThreads, kRing, s, a)
                          : art_stream::launch(art_append_scalar_kernel<T, LAYOUT>, dim3((unsigned)grid), kThreads, 0, s, a);
}

template <typename T>
cudaError_t launch_append(const AppendArgs &a, Way way, int grid, cudaStream_t s)
{
    if (way == kRows)
        return art_stream::launch(art_append_row_kernel<T>, dim3((unsigned)grid), kThreads, 0, s, a);
    return a.rope.layout == ART_ROPE_HALF ? launch_layout<T, ART_ROPE_HALF>(a, way, grid, s)
                                          : launch_layout<T, ART_ROPE_INTERLEAVED>(a, way, grid, s);
}

}  // namespace

extern "C" {

art_status_t art_rope_init_freqs(art_rope_t *rope, int32_t head_dim, int32_t rot_dim, int32_t layout,
                                 const double *inv_freq, double amplitude)
{
    if (!rope || (!inv_freq && rot_dim > 0))
        return ART_ERR_NULL;
    if (!head_size(head_dim))
        return ART_ERR_UNSUPPORTED;
    if ((layout != ART_ROPE_HALF && layout != ART_ROPE_INTERLEAVED) || !std::isfinite((float)amplitude))
        return ART_ERR_PARAM;
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2)
        return ART_ERR_PARAM;
    for (int i = 0; i < rot_dim / 2; ++i)
        if (!std::isfinite(inv_freq[i]))
            return ART_ERR_PARAM;
    std::memset(rope, 0, sizeof *rope);
    rope->head_dim = head_dim;
    rope->rot_dim = rot_dim;
    rope->layout = layout;
    rope->amplitude = (float)amplitude;
    for (int i = 0; i < rot_dim / 2; ++i) {
        // whole turns a position adds change nothing
        const long double turns = (long double)inv_freq[i] / 6.283185307179586476925286766559L;
        const long double frac = turns - floorl(turns);
        const long double fixed = roundl(frac * 0x1p64L);
        rope->turns[i] = fixed >= 0x1p64L ? 0 : (uint64_t)fixed;
    }
    return ART_OK;
}

art_status_t art_rope_init(art_rope_t *rope, int32_t head_dim, int32_t rot_dim, int32_t layout, double base,
                           int32_t scaling, double factor, int32_t original_len, double low_turns, double high_turns,
                           double amplitude)
{
    if (!rope)
        return ART_ERR_NULL;
    if (!head_size(head_dim))
        return ART_ERR_UNSUPPORTED;
    if (!(base > 1.0) || !std::isfinite(base) || scaling < ART_ROPE_SCALE_NONE || scaling > ART_ROPE_SCALE_BY_PARTS ||
        rot_dim < 0 || rot_dim > 2 * ART_ROPE_MAX_PAIRS)
        return ART_ERR_PARAM;
    if (scaling != ART_ROPE_SCALE_NONE && !(factor > 0.0 && std::isfinite(factor)))
        return ART_ERR_PARAM;
    if (scaling == ART_ROPE_SCALE_BY_PARTS &&
        (original_len <= 0 || !(high_turns > low_turns) || !std::isfinite(high_turns) || !std::isfinite(low_turns)))
        return ART_ERR_PARAM;
    double f[ART_ROPE_MAX_PAIRS];
    if (scaling == ART_ROPE_SCALE_NTK && rot_dim > 2)
        base *= std::pow(factor, (double)rot_dim / (rot_dim - 2.0));
    for (int i = 0; i < rot_dim / 2; ++i) {
        f[i] = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == ART_ROPE_SCALE_LINEAR)
            f[i] /= factor;
        if (scaling == ART_ROPE_SCALE_BY_PARTS) {
            const double turns = original_len * f[i] / 6.283185307179586476925286766559;
            double keep = (turns - low_turns) / (high_turns - low_turns);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f[i] = keep * f[i] + (1.0 - keep) * f[i] / factor;
        }
    }
    return art_rope_init_freqs(rope, head_dim, rot_dim, layout, f, amplitude);
}

art_status_t art_rope_append(const art_append_params_t *p, art_stream_t stream)
{
    if (!p || !p->rope)
        return ART_ERR_NULL;
    const art_tensor_t &q = p->q, &k = p->k, &v = p->v, &qo = p->q_out, &kc = p->k_cache, &vc = p->v_cache,
                       &pt = p->page_table, &sl = p->slots;
    if (q.ndim != 3 || k.ndim != 3 || v.ndim != 3 || qo.ndim != 3 || kc.ndim != 4 || vc.ndim != 4 || pt.ndim != 2 ||
        sl.ndim != 1 || (has(p->positions) && p->positions.ndim != 1) || (has(p->token_seq) && p->token_seq.ndim != 1) ||
        (has(p->mass) && p->mass.ndim != 3))
        return ART_ERR_SHAPE;
    const int64_t T = q.shape[0];
    if (T > 0 && (is_null(&q) || is_null(&k) || is_null(&v) || is_null(&qo) || is_null(&sl)))
        return ART_ERR_NULL;
    if (is_null(&kc) || is_null(&vc) || is_null(&pt))
        return ART_ERR_NULL;
    if ((q.dtype != ART_F32 && q.dtype != ART_BF16) || k.dtype != q.dtype || v.dtype != q.dtype || qo.dtype != q.dtype ||
        kc.dtype != q.dtype || vc.dtype != q.dtype || pt.dtype != ART_I32 || sl.dtype != ART_I32 ||
        (has(p->positions) && p->positions.dtype != ART_I32) || (has(p->token_seq) && p->token_seq.dtype != ART_I32) ||
        (has(p->mass) && p->mass.dtype != ART_F32))
        return ART_ERR_DTYPE;
    const int64_t Hq = q.shape[1], d = q.shape[2], Hkv = k.shape[1], B = pt.shape[0], mb = pt.shape[1];
    const int64_t NP = kc.shape[0], page = kc.shape[2];
    if (T < 0 || T > (int64_t)INT32_MAX / 2 || Hq <= 0 || Hq > 4096 || Hkv <= 0 || Hkv > 4096 || d <= 0 || B <= 0 ||
        B > (1 << 24) || mb <= 0 || NP <= 0 || NP > (int64_t)INT32_MAX || page <= 0 || page > 4096 ||
        mb * page > (int64_t)INT32_MAX - 4096)
        return ART_ERR_SHAPE;
    if (k.shape[0] != T || v.shape[0] != T || qo.shape[0] != T || sl.shape[0] != T || k.shape[2] != d || v.shape[2] != d ||
        qo.shape[1] != Hq || qo.shape[2] != d || v.shape[1] != Hkv || kc.shape[1] != Hkv || kc.shape[3] != d)
        return ART_ERR_SHAPE;
    for (int i = 0; i < 4; ++i)
        if (vc.shape[i] != kc.shape[i])
            return ART_ERR_SHAPE;
    if ((has(p->positions) && p->positions.shape[0] != T) || (has(p->token_seq) && p->token_seq.shape[0] != T) ||
        (!has(p->token_seq) && T > 0 && T != B))
        return ART_ERR_SHAPE;
    if (has(p->mass) && (p->mass.shape[0] != B || p->mass.shape[1] != Hkv || p->mass.shape[2] < mb * page))
        return ART_ERR_SHAPE;
    if (p->rope->head_dim != d)
        return ART_ERR_SHAPE;
    const art_rope_t &r = *p->rope;
    if (r.rot_dim < 0 || r.rot_dim > d || r.rot_dim % 2 || (r.layout != ART_ROPE_HALF && r.layout != ART_ROPE_INTERLEAVED) ||
        !head_size(d))
        return ART_ERR_PARAM;
    if (T == 0)
        return ART_OK;
    const int64_t es = elem_size(q.dtype);
    for (const art_tensor_t *t : {&q, &k, &v, &qo})
        if (t->stride[2] != 1 || !aligned(t->data, es) || t->stride[0] < 0 || t->stride[1] < 0)
            return ART_ERR_SHAPE;
    if (!apart(qo))
        return ART_ERR_SHAPE;
    // q_out may be q itself, rotated in place, but not q seen through other strides
    if (qo.data == q.data && (qo.stride[0] != q.stride[0] || qo.stride[1] != q.stride[1]))
        return ART_ERR_SHAPE;
    for (const art_tensor_t *t : {&kc, &vc}) {
        if (t->stride[3] != 1 || !aligned(t->data, 16) || !apart(*t))
            return ART_ERR_SHAPE;
        for (int i = 0; i < 3; ++i)
            if (t->stride[i] <= 0 || (t->stride[i] * es) % 16)
                return ART_ERR_SHAPE;
    }
    if (pt.stride[1] != 1 || pt.stride[0] < 0 || sl.stride[0] != 1 || (has(p->positions) && p->positions.stride[0] != 1) ||
        (has(p->token_seq) && p->token_seq.stride[0] != 1) || !aligned(pt.data, 4) || !aligned(sl.data, 4) ||
        !aligned(p->positions.data, 4) || !aligned(p->token_seq.data, 4) ||
        (p->device_status && !aligned(p->device_status, 4)))
        return ART_ERR_SHAPE;
    if (has(p->mass) && (!aligned(p->mass.data, 4) || p->mass.stride[2] != 1 || !apart(p->mass)))
        return ART_ERR_SHAPE;
    AppendArgs a;
    a.q = q.data;
    a.k = k.data;
    a.v = v.data;
    a.qo = qo.data;
    a.kc = kc.data;
    a.vc = vc.data;
    a.qs0 = q.stride[0];
    a.qs1 = q.stride[1];
    a.ks0 = k.stride[0];
    a.ks1 = k.stride[1];
    a.vs0 = v.stride[0];
    a.vs1 = v.stride[1];
    a.qos0 = qo.stride[0];
    a.qos1 = qo.stride[1];
    a.kc0 = kc.stride[0];
    a.kc1 = kc.stride[1];
    a.kc2 = kc.stride[2];
    a.vc0 = vc.stride[0];
    a.vc1 = vc.stride[1];
    a.vc2 = vc.stride[2];
    a.pt = static_cast<const int32_t *>(pt.data);
    a.pts0 = pt.stride[0];
    a.slots = static_cast<const int32_t *>(sl.data);
    a.pos = static_cast<const int32_t *>(p->positions.data);
    a.seq = static_cast<const int32_t *>(p->token_seq.data);
    a.mass = static_cast<float *>(p->mass.data);
    a.ms0 = p->mass.stride[0];
    a.ms1 = p->mass.stride[1];
    a.T = (int)T;
    a.B = (int)B;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.d = (int)d;
    a.page = (int)page;
    a.max_blocks = (int)mb;
    a.num_pages = (int)NP;
    a.status = p->device_status;
    a.rope = r;
    const int E = (int)(16 / es);
    const bool vectors = vector_rows(q, 3) && vector_rows(k, 3) && vector_rows(v, 3) && vector_rows(qo, 3);
    const Way way = !vectors ? kScalar : r.layout == ART_ROPE_INTERLEAVED || r.rot_dim % (2 * E) == 0 ? kPieces : kRows;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // Threads that share a token's heads: enough of them to give every SM two
    // CTAs, or at most one head each.  When the tokens alone fill the card, up to
    // four that have eight heads or more each to spend their sines on (28 + 4 heads
    // of 128, 453 MB: 71 us with four, 76 with one, whose loads are few; 8 + 1 heads of
    // 256, 254 MB: 76 us with four, 44 with one); the row kernel's warps each take a
    // whole token (94 us; 111 us with two to a token).
    const int64_t want = (int64_t)art_stream::sm_count() * 2 * kThreads;
    int64_t grid;
    int lanes = 1;
    if (way == kRows) {
        a.units = (int)(d / E);
        a.group = 1;
        while (a.group < 32 && a.group < a.units)
            a.group *= 2;
        while (lanes * (32 / a.group) < Hq + Hkv && T * lanes * 32 < want)
            lanes *= 2;
        grid = (T * lanes + kThreads / 32 - 1) / (kThreads / 32);
    } else {
        a.units = way == kPieces ? (int)(d / (2 * E)) : (int)(r.rot_dim / 2 + (d - r.rot_dim));
        while (lanes < 4 && Hq + Hkv >= lanes * 2 * 8)
            lanes *= 2;
        while (lanes * 2 * a.units <= kThreads && lanes < Hq + Hkv && T * a.units * lanes < want)
            lanes *= 2;
        const int64_t threads = T * a.units * lanes, cap = (int64_t)art_stream::sm_count() * 32;
        const int tpb = kThreads / (a.units * lanes);    // tokens a CTA
        grid = way == kPieces ? (T + tpb - 1) / tpb : (threads + kThreads - 1) / kThreads;
        if (way == kScalar && grid > cap)
            grid = cap;
    }
    a.lanes = lanes;
    const cudaError_t e = q.dtype == ART_BF16 ? launch_append<__nv_bfloat16>(a, way, (int)grid, s)
                                              : launch_append<float>(a, way, (int)grid, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return ART_ERR_LAUNCH;
    }
    return ART_OK;
}

}  // extern "C"
