// Attention of trees of drafted tokens over the 8-bit paged K/V cache (mrope_attend_tree_kv8).
//
//   out[t, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q[t, h] . k_j - max),
//
// over the positions j that query token i (of len) of a sequence of ctx positions sees: those before ctx - len,
// and ctx - len + b for the bits b that are set in its row of the mask.  Rows, tiles, chunks of contexts and the
// join are those of mrope_attend.h; a row is a (token, head of the group) pair, row = i * g + head.
//
// One workgroup: 16, 32 or 64 rows against a chunk of the context, its four waves taking 32 tokens in turn, each
// with all the rows.  S^T = K Q^T (16 x 16 x 32): a lane ends with the scores of one row of each sixteen (its
// column) for eight neighbouring tokens, which is just the operand that O^T = V^T P^T wants of P, so nothing moves
// between lanes and the waves meet only once, at the end.  A block's K and V are decoded once for all rows (codes
// are exact in 16 bits, V with its scale).  The queries wait in LDS in the order of the instruction's operand.
// P is taken in two bf16 terms for the 16-bit types and three for fp32, fp32 queries in three (each the bf16 nearest
// to what the terms before it leave).
//
// Only blocks that reach past ctx - len, or into a page that is not there, look at the mask.
#include <algorithm>

#include "mrope_attend.h"

namespace mrope {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kTreeWaves = kFewWaves;
template <int IO>
constexpr int kQTerms = IO == kIoF32 ? 3 : 1;
template <int IO>
constexpr int kPTerms = IO == kIoF32 ? 3 : 2;

template <int IO>
__device__ __forceinline__ f32x4 mfma_scores(u32x4 x, u32x4 y, f32x4 c)
{
    if constexpr (IO == kIoF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
}

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 x, u32x4 y, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
}

// Two e4m3 bytes of a key as the scores' 16-bit type (exact).  bf16 takes the page's scale at once; fp16 has no
// room for it, and the scores are multiplied instead.
template <int IO, bool HI>
__device__ __forceinline__ uint32_t key_pair(uint32_t u, float scale)
{
    if constexpr (IO == kIoF16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, HI));
    else return bf16_pair<HI>(u, scale);
}

template <int IO, int D, int NB>
struct alignas(16) TreeLds {
    union {
        u32x4 q[NB][kQTerms<IO>][D / 32][64];  // the operand's pieces by lane
        float o[kTreeWaves][16][D + 4];        // sixteen rows' parts, when the queries have done their work
    };
    float ml[kTreeWaves][16 * NB][2];
};

// Workgroups of a compute unit that the registers let run at once.
constexpr int tree_resident(int head_dim, int nb)
{
    const int r = head_dim * nb;
    return r >= 512 ? 1 : (r >= 256 ? 2 : (r >= 128 ? 3 : 4));
}

// V's page scale (2^8 smaller) beside which the running maximum follows at once.
constexpr float kLargeScale = 0x1p72f;

template <int IO, int D, int NB>
__global__ __launch_bounds__(64 * kTreeWaves, tree_resident(D, NB)) void attend_tree_kernel(AttendTree a, FewPlan p)
{
    constexpr int R = 16 * NB, QT = kQTerms<IO>, N = kPTerms<IO>;
    constexpr int NK = D / 64;   // 16-byte pieces of a key a lane holds
    constexpr int ND = D / 16;   // dims a lane's V operand holds of a token, and 16-dim tiles of O^T
    const Kv8 &kv = a.kv;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, grp = lane >> 4;
    const int g = a.nq / kv.nk, kvh = blockIdx.y;

    Cut cut = {0, 0, 0, 1};
    int32_t z = 0;
    Tile tl;
    if (p.max_cut == 0) {  // tables of one chunk
        if (!find_tile<R>(a, g, blockIdx.x, lane, tl)) return;
    } else {
        CutList *list = static_cast<CutList *>(a.workspace);
        int32_t rank, n_cut;
        const bool found = find_chunk<R>(a, g, blockIdx.x, p.budget, lane, cut, z, rank, n_cut);
        if (blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0) list->n = min(n_cut, p.max_cut);
        if (!found) return;
        if (cut.n > 1) {
            if (rank >= p.max_cut || cut.slot + cut.n > p.max_slots) return;  // (not for offsets that grow)
            if (z == 0 && kvh == 0 && threadIdx.x == 0) list->cut[rank] = cut;
        }
        make_tile<R>(a, g, cut.s, cut.tile, tl);
    }
    const int n_rows = min(R, tl.rows - tl.row0);
    const int32_t len = tl.rows / g;
    const int32_t seen = (int32_t)tl.seen, past = (int32_t)tl.past;  // (past >= -2^31: ctx >= 0)
    const int32_t open = min(max(past, 0), seen);                     // every row sees the positions before this
    const int32_t chunk = chunk_of(seen, cut.n, kFewUnit);
    const int32_t c0 = (int32_t)min((int64_t)z * chunk, (int64_t)seen), c1 = min(c0 + chunk, seen);

    __shared__ TreeLds<IO, D, NB> lds;

    // pages of this wave's half blocks from token `from` on, a lane each
    const int32_t *table = kv.tables + tl.s * kv.table_stride;
    int64_t base;
    float ks, vs;
    uint64_t valid_mask;
    auto look_up = [&](int32_t from) {
        base = 0;
        ks = vs = 1.0f;
        bool valid = false;
        const int64_t tok = (int64_t)from + ((lane >> 1) * kTreeWaves + wave) * 32 + (lane & 1) * 16;
        if (tok < c1) {
            const int32_t page = table[tok >> kv.bs_shift];
            valid = page >= 0 && page < kv.num_blocks;
            if (valid) {
                ks = kv.k_scale[(int64_t)page * kv.nk + kvh];
                vs = pow2(scale_exp_of(kv.v_scale[(int64_t)page * kv.nk + kvh]) - kVDown);  // (finite, whatever nobody sees)
                base = page * kv.c_block;
            }
            base += (tok & (kv.block_size - 1)) * kv.c_tok + kvh * kv.c_head;
        }
        valid_mask = __ballot(valid);
    };
    auto blocks_of = [&](int32_t from) {  // of this wave, in the tokens looked up from there
        const int n = (min(c1 - from, kFewPages) + 31) / 32;
        return n > wave ? (n - wave + kTreeWaves - 1) / kTreeWaves : 0;
    };
    look_up(c0);

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
    int n_mine = blocks_of(c0);
    if (n_mine > 0) {
        load_k(0);
        load_v(0);
    }

    // the queries: piece f of lane (col, grp) is dims 64 * (f / 2) + 16 * grp + 8 * (f % 2) .. + 7 of row col
    for (int e = threadIdx.x; e < NB * (D / 32) * 64; e += 64 * kTreeWaves) {
        const int el = e & 63, f = (e >> 6) % (D / 32), nb = (e >> 6) / (D / 32);
        const int r = nb * 16 + (el & 15);
        float x[8] = {};
        if (r < n_rows) {
            const int row = tl.row0 + r;
            unpack8<IO>(load8<IO>(a.q, (int64_t)(tl.t0 + row / g) * a.q_tok + (int64_t)(kvh * g + row % g) * a.q_head +
                                           64 * (f >> 1) + 16 * (el >> 4) + 8 * (f & 1)), x);
        }
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = pack16x2<IO == kIoF16 ? kIoF16 : kIoBF16>(x[2 * i], x[2 * i + 1]);
                if (t + 1 < QT) {
                    float lo, hi;
                    unpack16x2<kIoBF16>(w[i], lo, hi);
                    x[2 * i] -= lo;
                    x[2 * i + 1] -= hi;
                }
            }
            lds.q[nb][t][f][el] = w;
        }
    }
    __syncthreads();

    int32_t itok[NB];  // the query token of this lane's row of each sixteen
#pragma unroll
    for (int n = 0; n < NB; ++n) itok[n] = (tl.row0 + min(n * 16 + col, n_rows - 1)) / g;
    // Which of the tokens mine0 .. + 7 query token i sees: bit q for mine0 + q.
    auto sees = [&](int32_t i, int32_t mine0, bool ok) {
        const int32_t j = mine0 - past;  // (the tree's token at mine0)
        const uint64_t *row = a.mask + (int64_t)(tl.t0 + i) * a.mask_words;
        const int32_t w = j >> 6;
        auto word = [&](int32_t k) { return k < 0 ? ~0ull : (k < a.mask_words ? row[k] : 0ull); };
        uint64_t bits = word(w) >> (j & 63);
        if ((j & 63) > 56) bits |= word(w + 1) << (64 - (j & 63));
        const int32_t n = min(min(len - j, seen - mine0), 8);
        return n > 0 && ok ? (uint32_t)bits & ((1u << n) - 1) : 0u;
    };

    float m[NB], l[NB];
    f32x4 o[NB][ND];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        m[n] = kNoMax;
        l[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < ND; ++i) o[n][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    for (int32_t from = c0;;) {
        for (int it = 0; it < n_mine; ++it) {
            const int32_t tok0 = from + (it * kTreeWaves + wave) * 32;
            const float ks0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ks), 2 * it));
            const float ks1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ks), 2 * it + 1));
            const float kscale = col < 8 ? ks0 : ks1;
            const bool ok0 = (valid_mask >> (2 * it)) & 1, ok1 = (valid_mask >> (2 * it + 1)) & 1;
            int here = lane;  // (opaque: the queries stay in LDS and are read anew)
            asm volatile("" : "+v"(here));
            f32x4 sa[NB], sb[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) sa[n] = sb[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x4 fa = {key_pair<IO, false>(ka[k][2 * h], kscale), key_pair<IO, true>(ka[k][2 * h], kscale),
                                      key_pair<IO, false>(ka[k][2 * h + 1], kscale), key_pair<IO, true>(ka[k][2 * h + 1], kscale)};
                    const u32x4 fb = {key_pair<IO, false>(kb[k][2 * h], kscale), key_pair<IO, true>(kb[k][2 * h], kscale),
                                      key_pair<IO, false>(kb[k][2 * h + 1], kscale), key_pair<IO, true>(kb[k][2 * h + 1], kscale)};
#pragma unroll
                    for (int t = 0; t < QT; ++t)
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            const u32x4 q = lds.q[n][t][2 * k + h][here];
                            sa[n] = mfma_scores<IO>(fa, q, sa[n]);
                            sb[n] = mfma_scores<IO>(fb, q, sb[n]);
                        }
                }
            if (it + 1 < n_mine) load_k(it + 1);

            // this lane: a row of each sixteen against tokens tok0 + 8*grp + 0..7
            const float vs0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(vs), 2 * it));
            const float vs1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(vs), 2 * it + 1));
            const float vscale = grp < 2 ? vs0 : vs1;
            const bool edge = tok0 + 32 > open || !ok0 || !ok1;  // wave-uniform
            const int32_t mine0 = tok0 + 8 * grp;
            // the maximum moves only where it has grown by 2^8: until then p exceeds 1 and nothing is lost (but
            // beside large values, where the sums have no room for it, it moves at once)
            const float lag = fmaxf(vs0, vs1) >= kLargeScale ? 0.0f : 8.0f;
            uint32_t vis[NB];
            u32x4 pf[NB][N];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                float p[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    p[j] = sa[n][j];
                    p[4 + j] = sb[n][j];
                }
                if constexpr (IO == kIoF16) {
                    const float f = grp < 2 ? ks0 : ks1;
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] *= f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) p[j] *= a.scale_log2;
                vis[n] = 0xff;
                if (edge) {
                    vis[n] = sees(itok[n], mine0, grp < 2 ? ok0 : ok1);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (!(vis[n] >> j & 1)) p[j] = -__builtin_inff();
                }
                float mx = p[0];
#pragma unroll
                for (int j = 1; j < 8; ++j) mx = fmaxf(mx, p[j]);
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                if (__any(mx > m[n] + lag)) {
                    const float m_new = fmaxf(m[n], mx);
                    const float f = __builtin_amdgcn_exp2f(m[n] - m_new);
                    l[n] *= f;
#pragma unroll
                    for (int i = 0; i < ND; ++i) o[n][i] *= f;
                    m[n] = m_new;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    p[j] = __builtin_amdgcn_exp2f(p[j] - m[n]);
                    l[n] += p[j];
                }
#pragma unroll
                for (int t = 0; t < N; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t w = pack16x2<kIoBF16>(p[2 * j], p[2 * j + 1]);
                        pf[n][t][j] = w;
                        if (t + 1 < N) {
                            float lo, hi;
                            unpack16x2<kIoBF16>(w, lo, hi);
                            p[2 * j] -= lo;
                            p[2 * j + 1] -= hi;
                        }
                    }
            }

            // A NaN that some rows see and others do not, or that nobody sees, must not reach the product: there it
            // is left out, and the rows that see it are told.
            bool nan = false;
            if (edge) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int w = 0; w < ND / 4; ++w) nan |= any_nan(vr[j].w[w]);
                nan = __any(nan);
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
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            u32x4 mine;
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mine[j] = (vis[n] >> (2 * j) & 1 ? 0x3f80u : 0u) | (vis[n] >> (2 * j + 1) & 1 ? 0x3f800000u : 0u);
                            const f32x4 cnt = mfma_bf16(ind, mine, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                if (cnt[q] > 0.0f) o[n][4 * w + e][q] = __builtin_nanf("");
                        }
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
#pragma unroll
                    for (int t = 0; t < N; ++t)
#pragma unroll
                        for (int n = 0; n < NB; ++n) o[n][4 * w + e] = mfma_bf16(fv, pf[n][t], o[n][4 * w + e]);
                }
            }
            if (it + 1 < n_mine) load_v(it + 1);
        }
        if (c1 - from <= kFewPages) break;
        from += kFewPages;
        look_up(from);
        n_mine = blocks_of(from);
        if (n_mine > 0) {
            load_k(0);
            load_v(0);
        }
    }

    // the waves' parts meet in LDS, sixteen rows at a time
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        l[n] += __shfl_xor(l[n], 16);
        l[n] += __shfl_xor(l[n], 32);
        if (lane < 16) {
            lds.ml[wave][n * 16 + col][0] = m[n];
            lds.ml[wave][n * 16 + col][1] = l[n];
        }
    }
    const bool whole = cut.n == 1;
    Partial<D, R> *part = reinterpret_cast<Partial<D, R> *>(static_cast<char *>(a.workspace) + cut_list_bytes(p.max_cut)) +
                          ((int64_t)(cut.slot + z) * kv.nk + kvh);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        if (n * 16 >= n_rows) break;
        __syncthreads();  // the queries, or the sixteen rows before, have been read
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float *dst = &lds.o[wave][col][(grp * 4 + q) * ND];
#pragma unroll
            for (int i = 0; i < ND; i += 4)
                *reinterpret_cast<f32x4 *>(dst + i) = f32x4{o[n][i][q], o[n][i + 1][q], o[n][i + 2][q], o[n][i + 3][q]};
        }
        __syncthreads();
        for (int e = threadIdx.x; e < min(16, n_rows - n * 16) * (D / 8); e += 64 * kTreeWaves) {
            const int r16 = e / (D / 8), rr = n * 16 + r16, d = e % (D / 8) * 8;
            float mm = kNoMax, ll = 0.0f, y[8] = {};
#pragma unroll
            for (int w = 0; w < kTreeWaves; ++w) mm = fmaxf(mm, lds.ml[w][rr][0]);
#pragma unroll
            for (int w = 0; w < kTreeWaves; ++w) {
                const float f = __builtin_amdgcn_exp2f(lds.ml[w][rr][0] - mm);
                ll += lds.ml[w][rr][1] * f;
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] += lds.o[w][r16][d + i] * f;
            }
            if (whole) {
                const int rw = tl.row0 + rr;
                const int64_t tok = tl.t0 + rw / g;
                const int head = kvh * g + rw % g;
                const float inv = out_factor(ll);
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
}

// ------------------------------------------------------------------ launchers ------------------
struct TreePlan {
    int nb;         // sixteens of rows of a tile
    int64_t tiles, grid;
    FewPlan few;
    size_t bytes;   // of the workspace
};

TreePlan make_plan(int64_t n_tokens, int32_t n_seqs, int32_t nq, int32_t nk, int32_t head_dim, int32_t table_width, int32_t block_size)
{
    TreePlan p{};
    const int64_t g = nq / nk, cap = std::max<int64_t>(1, (int64_t)table_width * block_size);
    const int64_t seq_rows = (n_tokens * g + n_seqs - 1) / n_seqs;
    p.nb = seq_rows <= 16 ? 1 : (seq_rows <= 32 || head_dim == 256 ? 2 : 4);
    const int64_t rows = 16 * p.nb, most = (cap + kFewUnit - 1) / kFewUnit;
    p.tiles = n_tokens * g / rows + n_seqs;
    p.few.budget = std::max(1, 256 * tree_resident(head_dim, p.nb) / nk);
    p.grid = std::min(p.tiles + p.few.budget, p.tiles * most);
    if (most > 1) {
        p.few.max_cut = (int32_t)std::min<int64_t>(p.tiles, p.few.budget);
        p.few.max_slots = (int32_t)std::min<int64_t>(2 * p.few.budget, p.tiles * most);
        p.bytes = cut_list_bytes(p.few.max_cut) + (size_t)(rows * (head_dim + 2) * 4) * nk * (size_t)p.few.max_slots;
    }
    return p;
}

template <int IO, int D, int NB>
hipError_t launch_tree_nb(const AttendTree &a, const TreePlan &p, hipStream_t stream)
{
    constexpr int R = 16 * NB;
    attend_tree_kernel<IO, D, NB><<<dim3((unsigned)p.grid, a.kv.nk), 64 * kTreeWaves, 0, stream>>>(a, p.few);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.few.max_cut == 0) return e;
    attend_join_kernel<IO, D, R, 1><<<dim3((unsigned)p.few.max_cut, a.kv.nk, R), kJoinThreads, 0, stream>>>(a, 0, p.few.max_cut);
    return hipGetLastError();
}

template <int IO, int D>
hipError_t launch_tree_d(const AttendTree &a, hipStream_t stream)
{
    const TreePlan p = make_plan(a.n_tokens, a.n_seqs, a.nq, a.kv.nk, D, a.kv.table_width, a.kv.block_size);
    switch (p.nb) {
    case 1: return launch_tree_nb<IO, D, 1>(a, p, stream);
    case 2: return launch_tree_nb<IO, D, 2>(a, p, stream);
    default:
        if constexpr (D < 256) return launch_tree_nb<IO, D, 4>(a, p, stream);
        return hipErrorInvalidValue;  // (the plan has none)
    }
}

template <int IO>
hipError_t launch_tree_io(const AttendTree &a, hipStream_t stream)
{
    switch (a.head_dim) {
    case 64: return launch_tree_d<IO, 64>(a, stream);
    case 128: return launch_tree_d<IO, 128>(a, stream);
    default: return launch_tree_d<IO, 256>(a, stream);
    }
}

}  // namespace

size_t attend_tree_workspace_bytes(int64_t n_tokens, int32_t n_seqs, int32_t nq, int32_t nk, int32_t head_dim, int32_t table_width,
                                   int32_t block_size)
{
    return make_plan(n_tokens, n_seqs, nq, nk, head_dim, table_width, block_size).bytes;
}

hipError_t launch_attend_tree(const AttendTree &a, int io, hipStream_t stream)
{
    if (io == kIoBF16) return launch_tree_io<kIoBF16>(a, stream);
    if (io == kIoF16) return launch_tree_io<kIoF16>(a, stream);
    return launch_tree_io<kIoF32>(a, stream);
}

}  // namespace mrope
