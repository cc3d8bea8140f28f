// Attention over the 8-bit paged K/V cache (mrope_attend_kv8).
//
//   out[t, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q[t, h] . k_j - max),
//   k_j = code * scale of its page and head, v_j likewise,
//
// over the positions j <= ctx - len + i that query token i (of len) of a sequence of ctx tokens sees,
// with the running maximum and sum of a softmax: one pass over the cache.  The g = nq / nk query
// heads of a KV head share its keys, so a row below is a (token, head of the group) pair:
// row = i * g + head.
#include <algorithm>

#include "mrope_kv8.h"
#include "mrope_rotary.h"

namespace mrope {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kNoMax = -3.0e38f;  // the running maximum before any visible key

// ------------------------------------------------------------------ the work of a workgroup ----
struct Tile {
    int32_t s;          // sequence
    int32_t row0;       // first row of the tile within the sequence
    int32_t rows;       // rows of the sequence
    int32_t t0;         // first query token of the sequence in the call
    int64_t past;       // ctx - len: token i sees positions <= past + i
    int64_t seen;       // positions the sequence's tables can hold and its context has
};

// Tile w of R rows.  Sequence s begins at tile floor(cu[s] * g / R) + s: the key grows by at least
// ceil(rows / R) a sequence.
template <int R>
__device__ __forceinline__ bool find_tile(const Attend &a, int g, int64_t w, int lane, Tile &t)
{
    int64_t first;
    int32_t len = 1;
    if (a.cu) {
        int32_t lo = 0, hi = a.n_seqs;
        while (hi - lo > 1) {
            const int32_t step = (hi - lo + 63) / 64;
            const int32_t p = lo + lane * step;
            const bool le = p < hi && (int64_t)a.cu[min(p, a.n_seqs)] * g / R + p <= w;
            const int c = __builtin_popcountll(__ballot(le));
            hi = min(hi, lo + c * step);
            lo += (c - 1) * step;
        }
        t.s = __builtin_amdgcn_readfirstlane(lo);
        t.t0 = a.cu[t.s];
        len = (int32_t)min((int64_t)a.cu[t.s + 1], a.n_tokens) - t.t0;
        first = (int64_t)t.t0 * g / R + t.s;
    } else {
        const int32_t per = (g + R - 1) / R;
        t.s = (int32_t)(w / per);
        t.t0 = t.s;
        first = (int64_t)t.s * per;
    }
    t.rows = len * g;
    const int64_t row0 = (w - first) * R;
    if (row0 >= t.rows) return false;
    t.row0 = (int32_t)row0;
    const int64_t ctx = max(a.ctx[t.s], 0);
    t.past = ctx - len;
    t.seen = min(ctx, (int64_t)a.kv.table_width << a.kv.bs_shift);
    return true;
}

// Positions that the row sees: [0, row_limit), <= 0 for none.
__device__ __forceinline__ int64_t row_limit(const Tile &t, int g, int row) { return min(t.seen, t.past + row / g + 1); }

// ------------------------------------------------------------------ few rows -------------------
// One workgroup: R rows against a chunk of the context, its four waves taking 32 tokens in turn.
//
// Everything chains without moving data between lanes.  S^T = K Q^T (16 x 16 x 32, bf16): a lane
// ends with the scores of one row (its column) for four keys of two 16-key tiles; those eight are
// the tokens 8*(lane/16) + 0..7 of the block (the tiles take the keys in that order), just the
// operand that O^T = V^T P^T wants of P, and the lane's V operand is eight tokens by D/16
// neighbouring dims, which one row of 16 lanes loads as whole cache rows.  So the running maximum,
// the sum and the rescaling are one number a lane.
//
// The matrix instruction has 16 columns and few rows use them, so the idle ones carry precision for
// nothing: column t*R + r holds the t-th bf16 term of row r (x = x0 + x1 + x2, each term the bf16
// nearest to what is left), for Q and again for P.  Two terms are exact for bf16 and fp16 queries and
// keep P to 2^-16; three hold fp32.  The codes of K and V are exact in bf16, their scales (powers of
// two) applied by the conversion.
//
// Bound: the cache's bytes, 2*D a token and KV head.
template <int NT>
constexpr int kRowsOf = NT == 2 ? 8 : 4;
constexpr int kFewWaves = 4;
constexpr int kMinChunk = 128;   // a block of 32 tokens a wave
constexpr int kMaxChunk = 4096;  // a lane keeps the page of one 16-token half block

__device__ __forceinline__ float row_ror8(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128, 0xF, 0xF, false));
}
__device__ __forceinline__ float row_ror4(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x124, 0xF, 0xF, false));
}
// Sum of a row's terms over the columns that hold them.
template <int NT>
__device__ __forceinline__ float sum_terms(float x)
{
    x += row_ror8(x);
    if constexpr (NT == 3) x += row_ror4(x);
    return x;
}

// Term t of x (t is the lane's): the bf16 nearest to what the terms before it leave.
template <int NT>
__device__ __forceinline__ float term(float x, int t)
{
    const float h = (float)(__bf16)x;
    const float r = x - h;
    if constexpr (NT == 2) return t ? r : h;
    const float m = (float)(__bf16)r;
    return t == 0 ? h : (t == 1 ? m : (t == 2 ? r - m : 0.0f));  // a fourth group of columns stays empty
}

// Two e4m3 bytes (the low or the high pair of u) times a power of two, as bf16 (exact).
template <bool HI>
__device__ __forceinline__ uint32_t bf16_pair(uint32_t u, float scale)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, scale, HI));
}

__device__ __forceinline__ bool any_nan(uint32_t u)
{
    const uint32_t x = (u & 0x7f7f7f7fu) + 0x01010101u;  // a byte's top bit: its low seven were all ones
    return (x & 0x80808080u) != 0;
}

template <int D>
struct VRow {
    uint32_t w[D / 64];  // D/16 bytes
};

template <int D>
__device__ __forceinline__ VRow<D> load_vrow(const uint8_t *p)
{
    VRow<D> r;
    if constexpr (D == 256) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
    } else if constexpr (D == 128) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = x.x, r.w[1] = x.y;
    } else {
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
    return r;
}

template <int D, int R>
struct Partial {  // of a tile and chunk, in the workspace
    float ml[R][2];
    float o[R][D];
};

template <int IO>
__device__ __forceinline__ void store_out8(const Attend &a, int64_t off, const float (&y)[8])
{
    store8<IO>(a.out, off, pack8<IO>(y));
}

template <int IO, int D, int NT>
__global__ __launch_bounds__(64 * kFewWaves, 2) void attend_few_kernel(Attend a, int chunk, int n_chunks)
{
    constexpr int R = kRowsOf<NT>;
    constexpr int NK = D / 64;   // 16-byte pieces of a key a lane holds
    constexpr int ND = D / 16;   // dims a lane's V operand holds of a token, and 16-dim tiles of O^T
    const Kv8 &kv = a.kv;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, grp = lane >> 4;
    const int g = a.nq / kv.nk, kvh = blockIdx.y, z = blockIdx.z;

    Tile tl;
    if (!find_tile<R>(a, g, blockIdx.x, lane, tl)) return;
    const int n_rows = min(R, tl.rows - tl.row0);
    const int64_t lim_last = row_limit(tl, g, tl.row0 + n_rows - 1);  // the most that a row of the tile sees
    const int64_t lim_first = row_limit(tl, g, tl.row0);
    const int64_t c0 = (int64_t)z * chunk;
    if (z > 0 && c0 >= lim_last) return;
    const int64_t c1 = min(c0 + chunk, lim_last);

    // pages of this wave's half blocks, a lane each
    const int32_t *table = a.kv.tables + tl.s * kv.table_stride;
    int64_t base = 0;
    float ks = 1.0f, vs = 1.0f;
    bool valid = false;
    {
        const int64_t tok = c0 + ((lane >> 1) * kFewWaves + wave) * 32 + (lane & 1) * 16;
        if (tok < c1) {
            const int32_t page = table[tok >> kv.bs_shift];
            valid = page >= 0 && page < kv.num_blocks;
            if (valid) {
                ks = kv.k_scale[(int64_t)page * kv.nk + kvh];
                vs = kv.v_scale[(int64_t)page * kv.nk + kvh];
                base = page * kv.c_block;
            }
            base += (tok & (kv.block_size - 1)) * kv.c_tok + kvh * kv.c_head;
        }
    }
    const uint64_t valid_mask = __ballot(valid);

    // Q's terms: this lane's column is term `t` of row `r`
    const int t = col / R, r = col % R;
    const bool live = t < NT && r < n_rows;
    const int row = tl.row0 + min(r, n_rows - 1);
    const int64_t lim = row_limit(tl, g, row);
    bf16x8 qf[2 * NK];
    {
        const int64_t off = (int64_t)(tl.t0 + row / g) * a.q_tok + (int64_t)(kvh * g + row % g) * a.q_head;
#pragma unroll
        for (int k = 0; k < 2 * NK; ++k) {
            float x[8];
            unpack8<IO>(load8<IO>(a.q, off + (k >> 1) * 64 + grp * 16 + (k & 1) * 8), x);
#pragma unroll
            for (int e = 0; e < 8; ++e) qf[k][e] = (__bf16)(live ? term<NT>(x[e], t) : 0.0f);
        }
    }

    const int n_blocks = (int)((c1 - c0 + 31) / 32);
    const int n_mine = n_blocks > wave ? (n_blocks - wave + kFewWaves - 1) / kFewWaves : 0;

    u32x4 ka[NK], kb[NK];
    VRow<D> vr[8];
    const int key = (col >> 2) * 8 + (col & 3);  // the tiles' keys: this one, and four further
    auto half_base = [&](int i, int half) {
        const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)base, 2 * i + half);
        const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)base >> 32), 2 * i + half);
        return (int64_t)(((uint64_t)hi << 32) | lo);
    };
    auto load_k = [&](int i) {
        const int64_t b0 = half_base(i, 0), b1 = half_base(i, 1);
        const uint8_t *p = kv.k + (col < 8 ? b0 : b1) + (key & 15) * kv.c_tok + grp * 16;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            ka[k] = *reinterpret_cast<const u32x4 *>(p + 64 * k);
            kb[k] = *reinterpret_cast<const u32x4 *>(p + 4 * kv.c_tok + 64 * k);
        }
    };
    auto load_v = [&](int i) {
        const int64_t b0 = half_base(i, 0), b1 = half_base(i, 1);
        const uint8_t *p = kv.v + (grp < 2 ? b0 : b1) + (grp & 1) * 8 * kv.c_tok + col * ND;
#pragma unroll
        for (int j = 0; j < 8; ++j) vr[j] = load_vrow<D>(p + j * kv.c_tok);
    };

    float m = kNoMax, l = 0.0f;
    f32x4 o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    if (n_mine > 0) {
        load_k(0);
        load_v(0);
    }
    for (int it = 0; it < n_mine; ++it) {
        const int64_t tok0 = c0 + (int64_t)(it * kFewWaves + wave) * 32;
        const float ks0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ks), 2 * it));
        const float ks1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ks), 2 * it + 1));
        const float kscale = col < 8 ? ks0 : ks1;
        const bool ok0 = (valid_mask >> (2 * it)) & 1, ok1 = (valid_mask >> (2 * it + 1)) & 1;
        f32x4 sa = {0.0f, 0.0f, 0.0f, 0.0f}, sb = sa;
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 fa = {bf16_pair<false>(ka[k][2 * h], kscale), bf16_pair<true>(ka[k][2 * h], kscale),
                                  bf16_pair<false>(ka[k][2 * h + 1], kscale), bf16_pair<true>(ka[k][2 * h + 1], kscale)};
                const u32x4 fb = {bf16_pair<false>(kb[k][2 * h], kscale), bf16_pair<true>(kb[k][2 * h], kscale),
                                  bf16_pair<false>(kb[k][2 * h + 1], kscale), bf16_pair<true>(kb[k][2 * h + 1], kscale)};
                sa = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fa), qf[2 * k + h], sa, 0, 0, 0);
                sb = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb), qf[2 * k + h], sb, 0, 0, 0);
            }
        if (it + 1 < n_mine) load_k(it + 1);

        // this lane: row r against tokens tok0 + 8*grp + 0..7
        float p[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            p[j] = sum_terms<NT>(sa[j]) * a.scale_log2;
            p[4 + j] = sum_terms<NT>(sb[j]) * a.scale_log2;
        }
        const bool ragged = tok0 + 32 > lim_first || !ok0 || !ok1;  // wave-uniform
        const bool ok = grp < 2 ? ok0 : ok1;
        const int64_t mine0 = tok0 + 8 * grp;
        if (ragged) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (!ok || mine0 + j >= lim) p[j] = -__builtin_inff();
        }
        float mx = p[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) mx = fmaxf(mx, p[j]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        if (__any(mx > m)) {
            const float m_new = fmaxf(m, mx);
            const float f = __builtin_amdgcn_exp2f(m - m_new);
            l *= f;
#pragma unroll
            for (int i = 0; i < ND; ++i) o[i] *= f;
            m = m_new;
        }
        uint32_t pf[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] = __builtin_amdgcn_exp2f(p[j] - m);
            l += p[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) pf[j] = pack16x2<kIoBF16>(term<NT>(p[2 * j], t), term<NT>(p[2 * j + 1], t));
        const bf16x8 pb = __builtin_bit_cast(bf16x8, u32x4{pf[0], pf[1], pf[2], pf[3]});

        const float vs0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(vs), 2 * it));
        const float vs1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(vs), 2 * it + 1));
        const float vscale = grp < 2 ? vs0 : vs1;
        bool nan = false;
        if (ragged) {
            // what no row of the tile sees may hold anything: it must not reach the product
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool off = !ok || mine0 + j >= lim_last;
#pragma unroll
                for (int w = 0; w < ND / 4; ++w) {
                    if (off) vr[j].w[w] = 0;
                    nan |= any_nan(vr[j].w[w]);
                }
            }
            nan = __any(nan);
        }
        uint32_t nan_vis[4];
        if (nan) {  // rows that do see a NaN take it below; the others must not
#pragma unroll
            for (int j = 0; j < 4; ++j)
                nan_vis[j] = (ok && mine0 + 2 * j < lim ? 0x3f80u : 0u) | (ok && mine0 + 2 * j + 1 < lim ? 0x3f800000u : 0u);
        }
#pragma unroll
        for (int w = 0; w < ND / 4; ++w) {
            // bytes of two tokens side by side, then bf16 pairs (token 2j, token 2j + 1) of one dim
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo[j] = __builtin_amdgcn_perm(vr[2 * j + 1].w[w], vr[2 * j].w[w], 0x05010400u);
                hi[j] = __builtin_amdgcn_perm(vr[2 * j + 1].w[w], vr[2 * j].w[w], 0x07030602u);
            }
            if (nan) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    u32x4 ind;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t &b = e < 2 ? lo[j] : hi[j];
                        const int sh = (e & 1) * 16;
                        const uint32_t x = b >> sh;
                        const bool n0 = (x & 0x7fu) == 0x7fu, n1 = (x & 0x7f00u) == 0x7f00u;
                        ind[j] = (n0 ? 0x3f80u : 0u) | (n1 ? 0x3f800000u : 0u);
                        if (n0) b &= ~(0xffu << sh);
                        if (n1) b &= ~(0xff00u << sh);
                    }
                    const f32x4 cnt = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, ind),
                        __builtin_bit_cast(bf16x8, u32x4{nan_vis[0], nan_vis[1], nan_vis[2], nan_vis[3]}),
                        f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (cnt[q] > 0.0f) o[4 * w + e][q] = __builtin_nanf("");
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u32x4 fv;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b = e < 2 ? lo[j] : hi[j];
                    fv[j] = e & 1 ? bf16_pair<true>(b, vscale) : bf16_pair<false>(b, vscale);
                }
                o[4 * w + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fv), pb, o[4 * w + e], 0, 0, 0);
            }
        }
        if (it + 1 < n_mine) load_v(it + 1);
    }

    // the waves' parts meet in LDS
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    __shared__ float so[kFewWaves][R][D];
    __shared__ float sml[kFewWaves][R][2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float y[ND];
#pragma unroll
        for (int i = 0; i < ND; ++i) y[i] = sum_terms<NT>(o[i][q]);
        if (col < R) {
            float *dst = &so[wave][r][(grp * 4 + q) * ND];
#pragma unroll
            for (int i = 0; i < ND; ++i) dst[i] = y[i];
        }
    }
    if (lane < R) {
        sml[wave][r][0] = m;
        sml[wave][r][1] = l;
    }
    __syncthreads();
    const bool whole = n_chunks == 1 || lim_last <= chunk;
    Partial<D, R> *part = static_cast<Partial<D, R> *>(a.workspace) +
                          (((int64_t)blockIdx.x * kv.nk + kvh) * n_chunks + z);
    for (int e = threadIdx.x; e < n_rows * (D / 8); e += 64 * kFewWaves) {
        const int rr = e / (D / 8), d = e % (D / 8) * 8;
        float mm = kNoMax, ll = 0.0f, y[8] = {};
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) mm = fmaxf(mm, sml[w][rr][0]);
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(sml[w][rr][0] - mm);
            ll += sml[w][rr][1] * f;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] += so[w][rr][d + i] * f;
        }
        if (whole) {
            const int rw = tl.row0 + rr;
            const int64_t tok = tl.t0 + rw / g;
            const int head = kvh * g + rw % g;
            const float inv = ll > 0.0f ? 1.0f / ll : (ll == 0.0f ? 0.0f : ll);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = ll == 0.0f ? 0.0f : y[i] * inv;
            store_out8<IO>(a, tok * a.o_tok + head * a.o_head + d, y);
            if (a.lse && d == 0)
                a.lse[tok * a.nq + head] = ll == 0.0f ? -__builtin_inff() : 0.69314718055994531f * (mm + __log2f(ll));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) part->o[rr][d + i] = y[i];
            if (d == 0) {
                part->ml[rr][0] = mm;
                part->ml[rr][1] = ll;
            }
        }
    }
}

// Joins a tile's chunks: one workgroup a row, D/4 lanes over its dims and the rest over the chunks.
template <int IO, int D, int R>
__global__ __launch_bounds__(256) void attend_join_kernel(Attend a, int chunk, int n_chunks)
{
    const int g = a.nq / a.kv.nk, kvh = blockIdx.y, rr = blockIdx.z;
    Tile tl;
    if (!find_tile<R>(a, g, blockIdx.x, threadIdx.x & 63, tl)) return;
    const int n_rows = min(R, tl.rows - tl.row0);
    const int64_t lim_last = row_limit(tl, g, tl.row0 + n_rows - 1);
    if (rr >= n_rows || lim_last <= chunk) return;
    const int n = (int)((lim_last + chunk - 1) / chunk);
    const Partial<D, R> *part = static_cast<const Partial<D, R> *>(a.workspace) +
                                ((int64_t)blockIdx.x * a.kv.nk + kvh) * n_chunks;
    constexpr int LANES = D / 4, PARTS = 256 / LANES;
    const int d = threadIdx.x % LANES * 4, sub = threadIdx.x / LANES;
    float m = kNoMax, l = 0.0f;
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int z = sub; z < n; z += PARTS) {
        const float pm = part[z].ml[rr][0], pl = part[z].ml[rr][1];
        const f32x4 po = *reinterpret_cast<const f32x4 *>(&part[z].o[rr][d]);
        const float mn = fmaxf(m, pm), f0 = __builtin_amdgcn_exp2f(m - mn), f1 = __builtin_amdgcn_exp2f(pm - mn);
        l = l * f0 + pl * f1;
        y = y * f0 + po * f1;
        m = mn;
    }
    __shared__ float sm[PARTS][2];
    __shared__ f32x4 sy[PARTS][LANES];
    sy[sub][d / 4] = y;
    if (d == 0) {
        sm[sub][0] = m;
        sm[sub][1] = l;
    }
    __syncthreads();
    const int e = threadIdx.x;
    if (e >= D / 8) return;
    float mm = kNoMax, ll = 0.0f, r[8] = {};
#pragma unroll
    for (int p = 0; p < PARTS; ++p) mm = fmaxf(mm, sm[p][0]);
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        const float f = __builtin_amdgcn_exp2f(sm[p][0] - mm);
        ll += sm[p][1] * f;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] += sy[p][2 * e + (i >> 2)][i & 3] * f;
    }
    const int rw = tl.row0 + rr;
    const int64_t tok = tl.t0 + rw / g;
    const int head = kvh * g + rw % g;
    const float inv = 1.0f / ll;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = ll == 0.0f ? 0.0f : r[i] * inv;
    store_out8<IO>(a, tok * a.o_tok + head * a.o_head + 8 * e, r);
    if (a.lse && e == 0)
        a.lse[tok * a.nq + head] = ll == 0.0f ? -__builtin_inff() : 0.69314718055994531f * (mm + __log2f(ll));
}

// ------------------------------------------------------------------ launchers ------------------
struct Plan {
    int64_t tiles;
    int chunk, n_chunks;
    size_t bytes;
};

// Chunks of the context: as many workgroups as fill the device several times over (kFill), no chunk
// below 128 tokens (one block a wave) nor above 4,096 (the pages that a wave's lanes keep).
constexpr int64_t kFill = 2048;

Plan plan_few(int64_t n_tokens, int32_t n_seqs, int32_t nq, int32_t nk, int32_t head_dim, int io, bool one_token,
              int32_t table_width, int32_t block_size)
{
    Plan p{};
    const int R = io == kIoF32 ? kRowsOf<3> : kRowsOf<2>;
    const int g = nq / nk;
    p.tiles = one_token ? (int64_t)n_seqs * ((g + R - 1) / R) : n_tokens * g / R + n_seqs;
    const int64_t cap = std::max<int64_t>(1, (int64_t)table_width * block_size);
    int64_t chunk = kMinChunk;
    while (chunk < kMaxChunk && p.tiles * nk * ((cap + chunk - 1) / chunk) > kFill) chunk *= 2;
    p.chunk = (int)chunk;
    p.n_chunks = (int)((cap + chunk - 1) / chunk);
    p.bytes = p.n_chunks > 1 ? (size_t)p.tiles * nk * p.n_chunks * (size_t)(R * (head_dim + 2) * 4) : 0;
    return p;
}

template <int IO, int D>
hipError_t launch_attend_d(const Attend &a, hipStream_t stream)
{
    constexpr int NT = IO == kIoF32 ? 3 : 2;
    const Plan p = plan_few(a.n_tokens, a.n_seqs, a.nq, a.kv.nk, D, IO, a.cu == nullptr, a.kv.table_width, a.kv.block_size);
    attend_few_kernel<IO, D, NT><<<dim3((unsigned)p.tiles, a.kv.nk, p.n_chunks), 64 * kFewWaves, 0, stream>>>(a, p.chunk, p.n_chunks);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.n_chunks == 1) return e;
    attend_join_kernel<IO, D, kRowsOf<NT>><<<dim3((unsigned)p.tiles, a.kv.nk, kRowsOf<NT>), 256, 0, stream>>>(a, p.chunk, p.n_chunks);
    return hipGetLastError();
}

template <int IO>
hipError_t launch_attend_io(const Attend &a, hipStream_t stream)
{
    switch (a.head_dim) {
    case 64: return launch_attend_d<IO, 64>(a, stream);
    case 128: return launch_attend_d<IO, 128>(a, stream);
    default: return launch_attend_d<IO, 256>(a, stream);
    }
}

}  // namespace

size_t attend_workspace_bytes(int64_t n_tokens, int32_t n_seqs, int32_t nq, int32_t nk, int32_t head_dim, int io,
                              bool one_token, int32_t table_width, int32_t block_size)
{
    return plan_few(n_tokens, n_seqs, nq, nk, head_dim, io, one_token, table_width, block_size).bytes;
}

hipError_t launch_attend(const Attend &a, int io, hipStream_t stream)
{
    if (io == kIoBF16) return launch_attend_io<kIoBF16>(a, stream);
    if (io == kIoF16) return launch_attend_io<kIoF16>(a, stream);
    return launch_attend_io<kIoF32>(a, stream);
}

}  // namespace mrope
