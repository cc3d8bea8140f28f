// Rotary and append to the 8-bit paged K/V cache (mrope_apply_kv8, mrope_decode_kv8).
//
// One workgroup per page that the call writes: it holds the page's tokens of every KV head in
// registers, rotates K, takes the largest magnitude of each head's rows for the page's scale, and
// writes the e4m3 rows -- one pass over Q, K and V, no atomics, and no order to depend on.  A page
// that a sequence continues keeps its rows: where the new rows need a larger scale the workgroup
// re-codes them (it is the page's only writer).
//
// Thread layout: LPR lanes a row (16 at 256 dims, each lane two chunks of 8 dims half a row apart, so
// that a load instruction covers whole lines; 16 at 128 and 8 at 64 dims with one chunk), block_size
// rows.  The lanes of a row also rotate the token's Q heads, LPR/8 heads at a time in the eight-lane
// layout of mrope_rotary.h, which the first eight lanes' K chunks share.
//
// Bound: HBM.  At 8 Q + 2 KV heads of 256 bf16 dims a token moves 2,048 B of Q (rotated dims, in and
// out), 2,048 B of K and V in and 1,024 B out.  Measured: 64 sequences of 4,096 tokens 271 us, 1,345 MB at
// 4.97 TB/s (a dense copy reaches 6.5, the 16-bit cache write 6.07: the waves of a page wait for one another
// between its largest value and its codes); 37 ragged fp32 sequences, 92 MB, 28 us.  Several pages a
// workgroup, the next one's rows fetched ahead, took 395 us: fewer workgroups fit beside them.
#include <algorithm>

#include "mrope_kv8.h"
#include "mrope_rotary.h"

namespace mrope {
namespace {

// y = own * c + partner * ss, each output rounded once to fp32 (rotate_chunk's arithmetic).
template <int IO>
__device__ __forceinline__ void rotate8(const Raw8<IO> &own, const double (&c)[8], const double (&ss)[8], float (&y)[8])
{
    float x[8], p[8];
    unpack8<IO>(own, x);
    unpack8<IO>(swap_pair<IO>(own), p);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (float)__builtin_fma((double)x[e], c[e], (double)p[e] * ss[e]);
}

constexpr float kMaxFloat = 3.402823466e38f;

// Eight values under the scale whose reciprocal is f; what is not finite becomes NaN.  The codes are not
// read back by the launch: they carry the non-temporal hint.
__device__ __forceinline__ void store_codes(uint8_t *p, float (&v)[8], float f)
{
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fabsf(v[e]) <= kMaxFloat ? v[e] * f : __builtin_nanf("");
    const u32x2 b = {pack_e4m3(v[0], v[1], v[2], v[3]), pack_e4m3(v[4], v[5], v[6], v[7])};
    __builtin_nontemporal_store(b, reinterpret_cast<u32x2 *>(p));
}

// Largest s in [0, n) with cu[s]/bs + 2s <= w: a 64-ary search of the wave.  The key grows by at
// least 2 a sequence and by one more than the pages that its tokens can touch (t tokens that begin
// inside a page touch at most (t - 2)/bs + 2), so the workgroups [key(s), key(s+1)) cover sequence s.
__device__ __forceinline__ int32_t find_seq(const int32_t *cu, int32_t n, int shift, int64_t w, int lane)
{
    int32_t lo = 0, hi = n;
    while (hi - lo > 1) {
        const int32_t step = (hi - lo + 63) / 64;
        const int32_t p = lo + lane * step;
        const bool le = p < hi && ((int64_t)(cu[min(p, n)] >> shift) + 2 * (int64_t)p) <= w;
        const int c = __builtin_popcountll(__ballot(le));  // >= 1: key(lo) <= w
        hi = min(hi, lo + c * step);
        lo += (c - 1) * step;
    }
    return lo;
}

template <int D>
constexpr int kRowLanes = D == 64 ? 8 : 16;

template <int IO, int D, int BS>
__global__ __launch_bounds__(BS * kRowLanes<D>) void append_kernel(Append a, Rotary rot)
{
    constexpr int LPR = kRowLanes<D>;             // lanes a row
    constexpr int NV = D / 8 / LPR;               // chunks of 8 dims a lane holds of a row
    constexpr int kWaves = BS * LPR / 64;
    // (K or V, head) units held at a time: 1,024 threads have 128 registers; in fp32 four take 32.4 us and two
    // 30.5 on the 37 ragged sequences, in bf16 there is no difference
    constexpr int kUnits = kWaves > 8 || IO == kIoF32 ? 2 : 4;
    const Kv8 &kv = a.kv;
    const int lane = threadIdx.x & 63;
    const int row = threadIdx.x / LPR, l = threadIdx.x % LPR;

    // the page: sequence s, positions [p0, p1) of it, the first at token t0 of the call
    const int32_t s = __builtin_amdgcn_readfirstlane(find_seq(a.cu, a.n_seqs, kv.bs_shift, blockIdx.x, lane));
    const int64_t first = a.cu[s], len = min((int64_t)a.cu[s + 1], a.n_tokens) - first;
    const int32_t at = a.pos ? a.pos[s] : 0;
    const int64_t off = max(at, 0);  // (a negative one is no position: only Q is rotated)
    const int64_t pg = (off >> kv.bs_shift) + ((int64_t)blockIdx.x - ((first >> kv.bs_shift) + 2 * (int64_t)s));
    const int64_t p0 = max(off, pg << kv.bs_shift), p1 = min(off + len, (pg + 1) << kv.bs_shift);
    const int cnt = (int)max(p1 - p0, (int64_t)0);
    if (cnt == 0) return;
    const int64_t t0 = first + (p0 - off);
    const int held = (int)(p0 - (pg << kv.bs_shift));  // rows that the sequence already has in the page
    int32_t page = -1;
    if (at >= 0 && pg < kv.table_width) page = kv.tables[s * kv.table_stride + pg];
    const bool mine = row >= held && row < held + cnt;
    const int64_t t = t0 + (mine ? row - held : 0);  // a row without a token reads the first one's

    // this lane's chunks of a row: dims 8*chunk(i); the first eight lanes hold dims 0..63 in the
    // rotation's order (neighbour lanes are partners)
    const int l8 = l & 7;
    const int rot_d = 32 * (l8 & 1) + 8 * (l8 >> 1);
    const int dim0 = l < 8 ? rot_d : 8 * l;

    const int n_units = 2 * kv.nk;  // unit 2h: K of head h, 2h + 1: V
    Raw8<IO> x[kUnits][NV];
    auto load_units = [&](int u0) {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            if (u0 + u >= n_units) continue;
            const int h = (u0 + u) >> 1;
            const bool is_v = u & 1;
            const int64_t base = is_v ? t * a.v_tok + h * a.v_head : t * a.k_tok + h * a.k_head;
            x[u][0] = load8<IO>(is_v ? a.v : a.k, base + dim0);
            if constexpr (NV == 2) x[u][1] = load8<IO>(is_v ? a.v : a.k, base + 128 + 8 * l);
        }
    };
    load_units(0);

    // cos and sin of the token, eight frequencies a lane (both halves of a wider row alike)
    double c[8], ss[8];
    {
        const int32_t pt = a.planes[t], ph = a.planes[a.plane_stride + t], pw = a.planes[2 * a.plane_stride + t];
        pair_sincos(lane_freq<false>(rot, l8 >> 1, l8 & 1), pt, ph, pw, c, ss);
    }

    // Q in place, LPR/8 heads at a time, four loads in flight
    constexpr int QG = LPR / 8;
    for (int h0 = 0; h0 < a.nq; h0 += 4 * QG) {
        Raw8<IO> y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int h = min(h0 + i * QG + (l >> 3), a.nq - 1);
            y[i] = load8<IO>(a.q, t * a.q_tok + h * a.q_head + rot_d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int h = h0 + i * QG + (l >> 3);
            y[i] = rotate_chunk<IO>(y[i], c, ss);
            if (mine && h < a.nq) store8<IO>(a.q, t * a.q_tok + h * a.q_head + rot_d, y[i]);
        }
    }

    auto row_values = [&](int u, int i, float (&v)[8], const float (&turned)[8]) {
        unpack8<IO>(x[u][i], v);
        if (i == 0 && !(u & 1) && l < 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = turned[e];
        }
    };
    // (nothing above waits for the table: the rows are on their way before the page is known)
    if (page < 0 || page >= kv.num_blocks) return;
    __shared__ float part[2][kUnits][kWaves];
    for (int u0 = 0, par = 0; u0 < n_units; u0 += kUnits, par ^= 1) {
        if (u0) load_units(u0);
        // the rotated dims of K in fp32; everything else stays as it was loaded until it is coded
        float turned[(kUnits + 1) / 2][8];
        float top[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            top[u] = 0.0f;
            if (u0 + u >= n_units) continue;
            if (!(u & 1)) rotate8<IO>(x[u][0], c, ss, turned[u / 2]);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[8];
                row_values(u, i, v, turned[u / 2]);
                // a value that is not finite is stored as NaN and has no part in the scale
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float m = __builtin_fabsf(v[e]);
                    if (mine && m <= kMaxFloat) top[u] = fmaxf(top[u], m);
                }
            }
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) top[u] = fmaxf(top[u], __shfl_xor(top[u], o));
        }
        if (lane == 0) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u) part[par][u][threadIdx.x >> 6] = top[u];
        }
        __syncthreads();  // the other half of `part` is free again once every wave is past here
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            if (u0 + u >= n_units) continue;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) top[u] = fmaxf(top[u], part[par][u][w]);
            const int h = (u0 + u) >> 1;
            const bool is_v = u & 1;
            float *scale = (is_v ? kv.v_scale : kv.k_scale) + (int64_t)page * kv.nk + h;
            uint8_t *out = (is_v ? kv.v : kv.k) + (int64_t)page * kv.c_block + row * kv.c_tok + h * kv.c_head;
            int e = scale_exp_for(top[u]);
            if (held > 0) {
                const int was = scale_exp_of(*scale);
                if (e > was) {  // the rows already here go to the larger scale
                    if (row < held) {
                        const float f = pow2(max(was - e, -126));
                        uint2 *p = reinterpret_cast<uint2 *>(out + 8 * l);
                        *p = make_uint2(shift_e4m3(p->x, f), shift_e4m3(p->y, f));
                        if constexpr (NV == 2) {
                            p = reinterpret_cast<uint2 *>(out + 128 + 8 * l);
                            *p = make_uint2(shift_e4m3(p->x, f), shift_e4m3(p->y, f));
                        }
                    }
                } else {
                    e = was;
                }
            }
            if (mine) {
                const float f = pow2(-e);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float v[8];
                    row_values(u, i, v, turned[u / 2]);
                    store_codes(out + (i ? 128 + 8 * l : dim0), v, f);
                }
            }
            top[u] = pow2(e);
        }
        // every thread has read the old scales before one writes the new ones
        if (held > 0) __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
                if (u0 + u < n_units) ((u & 1) ? kv.v_scale : kv.k_scale)[(int64_t)page * kv.nk + ((u0 + u) >> 1)] = top[u];
        }
    }
}

// One new token a sequence: a wave a sequence, four a workgroup.  The wave holds 64/LPR units (K or V of
// a head) of its token at a time, and eight Q heads; a unit's largest magnitude is a reduction over its
// lanes, so nothing meets in LDS.  Bound: latency (position -> page -> scale -> store): 4,096 sequences
// 9.1 us, 21 MB.  With a page a workgroup, as above, they took 58 us, fifteen of sixteen rows idle.
template <int IO, int D>
__global__ __launch_bounds__(256) void append_one_kernel(Append a, Rotary rot)
{
    constexpr int LPR = kRowLanes<D>, NV = D / 8 / LPR, UPW = 64 / LPR;
    const Kv8 &kv = a.kv;
    const int lane = threadIdx.x & 63;
    const int32_t s = __builtin_amdgcn_readfirstlane((int32_t)(blockIdx.x * 4 + (threadIdx.x >> 6)));
    if (s >= a.n_seqs) return;
    const int64_t t = s;
    const int32_t pos = a.pos[s];
    const int32_t plane = pos - a.amount[s];
    const int row = pos & (kv.block_size - 1);  // the sequence holds the rows before it
    const int32_t pg = pos >> kv.bs_shift;
    int64_t page = -1;
    if (pos >= 0 && pg < kv.table_width) page = kv.tables[s * kv.table_stride + pg];
    const bool write = page >= 0 && page < kv.num_blocks;

    const int l = lane % LPR, unit = lane / LPR, l8 = l & 7;
    const int rot_d = 32 * (l8 & 1) + 8 * (l8 >> 1);
    const int dim0 = l < 8 ? rot_d : 8 * l;
    const int n_units = 2 * kv.nk;  // unit 2h: K of head h, 2h + 1: V
    Raw8<IO> x[NV], y;
    auto load_unit = [&](int u) {
        const int h = min(u, n_units - 1) >> 1;
        const bool is_v = u & 1;
        const int64_t base = is_v ? t * a.v_tok + h * a.v_head : t * a.k_tok + h * a.k_head;
        x[0] = load8<IO>(is_v ? a.v : a.k, base + dim0);
        if constexpr (NV == 2) x[1] = load8<IO>(is_v ? a.v : a.k, base + 128 + 8 * l);
    };
    load_unit(unit);
    if (a.nq > 0) y = load8<IO>(a.q, t * a.q_tok + min(lane >> 3, a.nq - 1) * a.q_head + rot_d);
    double c[8], ss[8];
    pair_sincos(lane_freq<false>(rot, l8 >> 1, l8 & 1), plane, plane, plane, c, ss);
    for (int h0 = 0; h0 < a.nq; h0 += 8) {
        const int h = h0 + (lane >> 3);
        if (h0) y = load8<IO>(a.q, t * a.q_tok + min(h, a.nq - 1) * a.q_head + rot_d);
        y = rotate_chunk<IO>(y, c, ss);
        if (h < a.nq) store8<IO>(a.q, t * a.q_tok + h * a.q_head + rot_d, y);
    }
    if (!write) return;
    for (int u0 = 0; u0 < n_units; u0 += UPW) {
        const int u = u0 + unit;
        if (u0) load_unit(u);
        float v[NV][8], top = 0.0f;
        unpack8<IO>(x[0], v[0]);
        {
            float r[8];
            rotate8<IO>(x[0], c, ss, r);
            if (l < 8 && !(u & 1)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[0][e] = r[e];
            }
        }
        if constexpr (NV == 2) unpack8<IO>(x[1], v[1]);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float m = __builtin_fabsf(v[i][e]);
                if (m <= kMaxFloat) top = fmaxf(top, m);
            }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        if (u >= n_units) continue;
        const int h = u >> 1;
        float *scale = ((u & 1) ? kv.v_scale : kv.k_scale) + page * kv.nk + h;
        uint8_t *first = ((u & 1) ? kv.v : kv.k) + page * kv.c_block + h * kv.c_head;
        int e = scale_exp_for(top);
        if (row > 0) {
            const int was = scale_exp_of(*scale);
            if (e > was) {  // the rows already here go to the larger scale
                const float f = pow2(max(was - e, -126));
                for (int r0 = 0; r0 < row; r0 += 8) {  // eight rows a round trip
                    uint2 w[8][NV];
#pragma unroll
                    for (int r = 0; r < 8; ++r)
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            w[r][i] = *reinterpret_cast<const uint2 *>(first + min(r0 + r, row - 1) * kv.c_tok + 128 * i + 8 * l);
#pragma unroll
                    for (int r = 0; r < 8; ++r)
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            if (r0 + r < row)
                                *reinterpret_cast<uint2 *>(first + (r0 + r) * kv.c_tok + 128 * i + 8 * l) =
                                    make_uint2(shift_e4m3(w[r][i].x, f), shift_e4m3(w[r][i].y, f));
                }
            } else {
                e = was;
            }
        }
        const float f = pow2(-e);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            store_codes(first + row * kv.c_tok + (i ? 128 + 8 * l : dim0), v[i], f);
        if (l == 0) *scale = pow2(e);  // (every lane of the unit has read it)
    }
}

template <int IO, int D, int BS>
hipError_t launch_append_bs(const Append &a, const Rotary &r, hipStream_t stream)
{
    const int64_t blocks = (a.n_tokens >> a.kv.bs_shift) + 2 * (int64_t)a.n_seqs;
    append_kernel<IO, D, BS><<<dim3((unsigned)blocks), dim3(BS * kRowLanes<D>), 0, stream>>>(a, r);
    return hipGetLastError();
}

template <int IO, int D>
hipError_t launch_append_d(const Append &a, const Rotary &r, hipStream_t stream)
{
    if (!a.planes) {
        append_one_kernel<IO, D><<<dim3((unsigned)((a.n_seqs + 3) / 4)), 256, 0, stream>>>(a, r);
        return hipGetLastError();
    }
    switch (a.kv.block_size) {
    case 16: return launch_append_bs<IO, D, 16>(a, r, stream);
    case 32: return launch_append_bs<IO, D, 32>(a, r, stream);
    default: return launch_append_bs<IO, D, 64>(a, r, stream);
    }
}

template <int IO>
hipError_t launch_append_io(const Append &a, const Rotary &r, hipStream_t stream)
{
    switch (a.head_dim) {
    case 64: return launch_append_d<IO, 64>(a, r, stream);
    case 128: return launch_append_d<IO, 128>(a, r, stream);
    default: return launch_append_d<IO, 256>(a, r, stream);
    }
}

}  // namespace

hipError_t launch_append(const Append &a, const Rotary &r, int io, hipStream_t stream)
{
    if (io == kIoBF16) return launch_append_io<kIoBF16>(a, r, stream);
    if (io == kIoF16) return launch_append_io<kIoF16>(a, r, stream);
    return launch_append_io<kIoF32>(a, r, stream);
}

}  // namespace mrope
