// Element I/O and the lane-level rotation shared by the rotary kernels and the 8-bit cache append.
#pragma once

#include "mrope_internal.h"
#include "mrope_math.h"

namespace mrope {
namespace {

// ------------------------------------------------------------------ element I/O ----------------
// Element types of Q/K (the C ABI's dtype codes).
constexpr int kIoF32 = 0, kIoBF16 = 1, kIoF16 = 2;

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Two fp32 values to a packed pair of the 16-bit type, each rounded to nearest even.
template <int IO>
__device__ __forceinline__ uint32_t pack16x2(float a, float b)
{
    const f32x2_t f = {a, b};
    if constexpr (IO == kIoBF16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2_t));
}

// A packed pair of the 16-bit type to fp32 (exact).
template <int IO>
__device__ __forceinline__ void unpack16x2(uint32_t u, float &lo, float &hi)
{
    if constexpr (IO == kIoBF16) {
        lo = __uint_as_float(u << 16);
        hi = __uint_as_float(u & 0xffff0000u);
    } else {
        const f32x2_t f = __builtin_convertvector(__builtin_bit_cast(f16x2_t, u), f32x2_t);
        lo = f[0];
        hi = f[1];
    }
}

// 8 consecutive elements as raw 16-byte words: one for the 16-bit types, two for fp32.
template <int IO>
struct Raw8 {
    uint4 w[IO == kIoF32 ? 2 : 1];
};

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// Q, K and V chunks are read once: loads carry the non-temporal hint.  Measured on the 64 x 4096
// workload: mrope_apply 119 -> 113 us, mrope_apply_ids 124 -> 117 us back to back, and no slower
// from cold caches; marking the stores as well made both slower.
__device__ __forceinline__ uint4 load16_nt(const void *p)
{
    const u32x4_t v = __builtin_nontemporal_load(static_cast<const u32x4_t *>(p));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

template <int IO>
__device__ __forceinline__ Raw8<IO> load8(const void *base, int64_t elem)
{
    Raw8<IO> r;
    if constexpr (IO != kIoF32) {
        r.w[0] = load16_nt(static_cast<const uint16_t *>(base) + elem);
    } else {
        const float *p = static_cast<const float *>(base) + elem;
        r.w[0] = load16_nt(p);
        r.w[1] = load16_nt(p + 4);
    }
    return r;
}

template <int IO>
__device__ __forceinline__ void store8(void *base, int64_t elem, const Raw8<IO> &r)
{
    if constexpr (IO != kIoF32) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + elem) = r.w[0];
    } else {
        uint4 *p = reinterpret_cast<uint4 *>(static_cast<float *>(base) + elem);
        p[0] = r.w[0];
        p[1] = r.w[1];
    }
}

// A store into another buffer than the one read (a cache row, an out-of-place head) is not read
// back by the launch: it carries the non-temporal hint.  Measured on 64 x 4096 bf16 tokens: the
// fused K/V cache write 335 -> 281 us, mrope_apply_kv 328 -> 272 us; a 4,096-sequence decode step
// 7.4 -> 6.7 us (out of place: see copy_rest_kernel).  In-place stores
// take the hint only when the launch writes more in place than the memory-side cache absorbs
// (the fixed-head kernels' NTS argument, chosen by the host).
template <int IO>
__device__ __forceinline__ void store8_nt(void *base, int64_t elem, const Raw8<IO> &r)
{
    u32x4_t *p;
    if constexpr (IO != kIoF32) p = reinterpret_cast<u32x4_t *>(static_cast<uint16_t *>(base) + elem);
    else p = reinterpret_cast<u32x4_t *>(static_cast<float *>(base) + elem);
#pragma unroll
    for (int i = 0; i < (IO == kIoF32 ? 2 : 1); ++i)
        __builtin_nontemporal_store((u32x4_t){r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w}, p + i);
}

// Non-temporal or plain store, chosen at compile time: with a run-time choice the compiler merges
// the two stores of the branches into one plain store (the hint is lost).
template <int IO, bool NT>
__device__ __forceinline__ void store8_as(void *base, int64_t elem, const Raw8<IO> &r)
{
    if constexpr (NT) store8_nt<IO>(base, elem, r);
    else store8<IO>(base, elem, r);
}

template <int IO>
__device__ __forceinline__ void unpack8(const Raw8<IO> &r, float (&x)[8])
{
    if constexpr (IO != kIoF32) {
        const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack16x2<IO>(u[i], x[2 * i], x[2 * i + 1]);
    } else {
        const uint32_t u[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    }
}

template <int IO>
__device__ __forceinline__ Raw8<IO> pack8(const float (&y)[8])
{
    Raw8<IO> r;
    if constexpr (IO != kIoF32) {
        r.w[0] = make_uint4(pack16x2<IO>(y[0], y[1]), pack16x2<IO>(y[2], y[3]), pack16x2<IO>(y[4], y[5]),
                            pack16x2<IO>(y[6], y[7]));
    } else {
        r.w[0] = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
        r.w[1] = make_uint4(__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]), __float_as_uint(y[7]));
    }
    return r;
}

// ------------------------------------------------------------------ rotary ---------------------
// Lane layout: eight lanes per token.  Lane l = 2m + half holds the 8 consecutive dims
// [32*half + 8m, 32*half + 8m + 8) of a head: frequencies j = 8m .. 8m+7, the x_j side (half 0) or
// the x_{j+32} side (half 1).  The eight lanes of a token cover one whole 128-byte line per head
// (bf16) with one load instruction, and rotate-half partners are neighbour lanes (l, l^1), which
// swap their data with one DPP move per dword.

// Value of the neighbour lane (l ^ 1) by DPP quad_perm [1,0,3,2].
__device__ __forceinline__ uint32_t swap_pair(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);
}
__device__ __forceinline__ double swap_pair(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = swap_pair((uint32_t)u), hi = swap_pair((uint32_t)(u >> 32));
    return __builtin_bit_cast(double, lo | (hi << 32));
}
template <int IO>
__device__ __forceinline__ Raw8<IO> swap_pair(const Raw8<IO> &r)
{
    Raw8<IO> o;
#pragma unroll
    for (int k = 0; k < (IO == kIoF32 ? 2 : 1); ++k)
        o.w[k] = make_uint4(swap_pair(r.w[k].x), swap_pair(r.w[k].y), swap_pair(r.w[k].z), swap_pair(r.w[k].w));
    return o;
}

// The four inverse frequencies a lane evaluates (half 0: 8m..8m+3, half 1: 8m+4..8m+7) and the
// plane each reads, 2 bits apiece.  kSelect: taken from the kernel arguments by uniform selects, for
// kernels that read them once before a token loop -- a lane-dependent index into the argument block
// is a vector memory load, and inside the loop the wait for it would also wait for the prefetched
// Q/K loads.  Otherwise (decode: one token, no prefetch) that indexed load is the cheaper form: it
// travels with the data load and needs no registers for all 32 values.
struct LaneFreq {
    float f[4];
    uint32_t sel;
    int half;
};

template <bool kSelect>
__device__ __forceinline__ LaneFreq lane_freq(const Rotary &rot, int m, int half)
{
    LaneFreq r;
    const int q = 2 * m + half;  // j0 = 4q
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kSelect) {
            float v = 0.0f;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                float x = rot.inv_freq[4 * t + i];
                asm volatile("" : "+s"(x));  // keep the selects: no indexed reload of the argument block
                v = q == t ? x : v;
            }
            r.f[i] = v;
        } else {
            r.f[i] = rot.inv_freq[4 * q + i];
        }
    }
    r.sel = (uint32_t)(rot.plane_sel >> (8 * q));
    r.half = half;
    return r;
}

// (cos, sign*sin) of frequencies 8m .. 8m+7 for lane pair m.  Each lane evaluates its four and the
// pair swaps results.  ss = -sin on the x_j side and +sin on the x_{j+32} side, so every output is
// y = own*c + partner*ss.
__device__ __forceinline__ void pair_sincos(const LaneFreq &lf, int32_t pt, int32_t ph, int32_t pw, double (&c)[8],
                                            double (&ss)[8])
{
    const int half = lf.half;
    double oc[4], os[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pl = (lf.sel >> (2 * i)) & 3u;
        const int32_t pos = pl == 1u ? ph : (pl == 2u ? pw : pt);
        const float a = (float)pos * lf.f[i];
        sincos_angle(a, &os[i], &oc[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double pc = swap_pair(oc[i]), ps = swap_pair(os[i]);
        c[i] = half ? pc : oc[i];
        c[4 + i] = half ? oc[i] : pc;
        const double s_lo = half ? ps : os[i], s_hi = half ? os[i] : ps;
        ss[i] = half ? s_lo : -s_lo;
        ss[4 + i] = half ? s_hi : -s_hi;
    }
}

// One head chunk: own holds this lane's 8 dims, the partner's come by DPP.
template <int IO>
__device__ __forceinline__ Raw8<IO> rotate_chunk(const Raw8<IO> &own, const double (&c)[8], const double (&ss)[8])
{
    float x[8], p[8], y[8];
    unpack8<IO>(own, x);
    unpack8<IO>(swap_pair<IO>(own), p);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (float)__builtin_fma((double)x[e], c[e], (double)p[e] * ss[e]);
    return pack8<IO>(y);
}

}  // namespace
}  // namespace mrope
