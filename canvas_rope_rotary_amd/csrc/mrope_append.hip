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
// out), 2,048 B of K and V in and 1,024 B out.
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
    constexpr int kUnits = kWaves > 8 ? 2 : 4;    // (K or V, head) units held at a time: 1,024 threads have 128 registers
    const Kv8 &kv = a.kv;
    const int lane = threadIdx.x & 63;
    const int row = threadIdx.x / LPR, l = threadIdx.x % LPR;

    // the page: sequence s, positions [p0, p1) of it, the first at token t0 of the call
    int32_t s;
    int64_t p0, p1, t0, pg;
    bool write = true;
    if (a.planes) {
        s = __builtin_amdgcn_readfirstlane(find_seq(a.cu, a.n_seqs, kv.bs_shift, blockIdx.x, lane));
        const int64_t first = a.cu[s], len = min((int64_t)a.cu[s + 1], a.n_tokens) - first;
        int64_t off = a.pos ? a.pos[s] : 0;
        if (off < 0) {  // no such position: only Q is rotated
            write = false;
            off = 0;
        }
        pg = (off >> kv.bs_shift) + ((int64_t)blockIdx.x - ((first >> kv.bs_shift) + 2 * (int64_t)s));
        p0 = max(off, pg << kv.bs_shift);
        p1 = min(off + len, (pg + 1) << kv.bs_shift);
        t0 = first + (p0 - off);
    } else {
        s = blockIdx.x;
        p0 = a.pos[s];
        t0 = s;
        if (p0 < 0) {
            write = false;
            p0 = 0;
        }
        p1 = p0 + 1;
        pg = p0 >> kv.bs_shift;
    }
    const int cnt = (int)(p1 - p0);
    if (cnt <= 0) return;
    const int held = (int)(p0 - (pg << kv.bs_shift));  // rows that the sequence already has in the page
    int64_t page = -1;
    if (write && kv.nk > 0 && pg < kv.table_width) page = kv.tables[s * kv.table_stride + pg];
    write = page >= 0 && page < kv.num_blocks;

    const bool mine = row >= held && row < held + cnt;
    const int64_t t = t0 + (mine ? row - held : 0);  // a row without a token reads the first one's

    // this lane's chunks of a row: dims 8*chunk(i); the first eight lanes hold dims 0..63 in the
    // rotation's order (neighbour lanes are partners)
    const int l8 = l & 7;
    const int rot_d = 32 * (l8 & 1) + 8 * (l8 >> 1);
    const int dim0 = l < 8 ? rot_d : 8 * l;

    const int n_units = write ? 2 * kv.nk : 0;  // unit 2h: K of head h, 2h + 1: V
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
        int32_t pt, ph, pw;
        if (a.planes) {
            pt = a.planes[t];
            ph = a.planes[a.plane_stride + t];
            pw = a.planes[2 * a.plane_stride + t];
        } else {
            pt = ph = pw = a.pos[s] - a.amount[s];
        }
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

    __shared__ float part[2][kUnits][kWaves];
    for (int u0 = 0, par = 0; u0 < n_units; u0 += kUnits, par ^= 1) {
        if (u0) load_units(u0);
        float y[kUnits][NV][8];
        float top[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            top[u] = 0.0f;
            if (u0 + u >= n_units) continue;
            if (u & 1) {
                unpack8<IO>(x[u][0], y[u][0]);
            } else {
                float r[8];
                unpack8<IO>(x[u][0], y[u][0]);
                rotate8<IO>(x[u][0], c, ss, r);
                if (l < 8) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[u][0][e] = r[e];
                }
            }
            if constexpr (NV == 2) unpack8<IO>(x[u][1], y[u][1]);
            // a value that is not finite is stored as NaN and has no part in the scale
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float m = __builtin_fabsf(y[u][i][e]);
                    const bool ok = m <= 3.402823466e38f;
                    if (mine && ok) top[u] = fmaxf(top[u], m);
                    if (!ok) y[u][i][e] = __builtin_nanf("");
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
            float *scale = (is_v ? kv.v_scale : kv.k_scale) + page * kv.nk + h;
            uint8_t *out = (is_v ? kv.v : kv.k) + page * kv.c_block + row * kv.c_tok + h * kv.c_head;
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
                    const uint2 b = make_uint2(
                        pack_e4m3(y[u][i][0] * f, y[u][i][1] * f, y[u][i][2] * f, y[u][i][3] * f),
                        pack_e4m3(y[u][i][4] * f, y[u][i][5] * f, y[u][i][6] * f, y[u][i][7] * f));
                    *reinterpret_cast<uint2 *>(out + (i ? 128 + 8 * l : dim0)) = b;
                }
            }
            top[u] = pow2(e);
        }
        // every thread has read the old scales before one writes the new ones
        if (held > 0) __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
                if (u0 + u < n_units) ((u & 1) ? kv.v_scale : kv.k_scale)[page * kv.nk + ((u0 + u) >> 1)] = top[u];
        }
    }
}

template <int IO, int D, int BS>
hipError_t launch_append_bs(const Append &a, const Rotary &r, hipStream_t stream)
{
    const int64_t blocks = a.planes ? (a.n_tokens >> a.kv.bs_shift) + 2 * (int64_t)a.n_seqs : a.n_seqs;
    append_kernel<IO, D, BS><<<dim3((unsigned)blocks), dim3(BS * kRowLanes<D>), 0, stream>>>(a, r);
    return hipGetLastError();
}

template <int IO, int D>
hipError_t launch_append_d(const Append &a, const Rotary &r, hipStream_t stream)
{
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
