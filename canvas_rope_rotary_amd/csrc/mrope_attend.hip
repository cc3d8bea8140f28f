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

// V is decoded 2^8 smaller than it is and the output divided by l / 2^8: a code times its scale can pass
// fp32's largest value (448 * 2^120), and the sums have as much room above it; the smallest, 2^-9 * 2^-96, stays far above
// the smallest normal bf16.
constexpr int kVDown = 8;
constexpr float kVUp = 256.0f;

__device__ __forceinline__ float out_factor(float l) { return l == 0.0f ? 0.0f : kVUp / l; }

// ------------------------------------------------------------------ the work of a workgroup ----
struct Tile {
    int32_t s;          // sequence
    int32_t row0;       // first row of the tile within the sequence
    int32_t rows;       // rows of the sequence
    int32_t t0;         // first query token of the sequence in the call
    int64_t past;       // ctx - len: token i sees positions <= past + i
    int64_t seen;       // positions the sequence's tables can hold and its context has
};

// Tile k of R rows of sequence s, whose first token is t0 of len.
template <int R>
__device__ __forceinline__ bool make_tile(const Attend &a, int g, int32_t s, int32_t t0, int32_t len, int64_t k, Tile &t)
{
    t.s = s;
    t.t0 = t0;
    t.rows = len * g;
    if (k < 0 || k * R >= t.rows) return false;
    t.row0 = (int32_t)k * R;
    const int64_t ctx = max(a.ctx[s], 0);
    t.past = ctx - len;
    t.seen = min(ctx, (int64_t)a.kv.table_width << a.kv.bs_shift);
    return true;
}

template <int R>
__device__ __forceinline__ bool make_tile(const Attend &a, int g, int32_t s, int64_t k, Tile &t)
{
    if (!a.cu) return make_tile<R>(a, g, s, s, 1, k, t);
    const int32_t t0 = a.cu[s];
    return make_tile<R>(a, g, s, t0, (int32_t)min((int64_t)a.cu[s + 1], a.n_tokens) - t0, k, t);
}

// Tile w of R rows.  Sequence s begins at tile floor(cu[s] * g / R) + s: the key grows by at least
// ceil(rows / R) a sequence.
template <int R>
__device__ __forceinline__ bool find_tile(const Attend &a, int g, int64_t w, int lane, Tile &t)
{
    if (!a.cu) {
        const int32_t per = (g + R - 1) / R;
        const int32_t s = (int32_t)(w / per);
        return make_tile<R>(a, g, s, w - (int64_t)s * per, t);
    }
    int32_t lo = 0, hi = a.n_seqs;
    while (hi - lo > 1) {
        const int32_t step = (hi - lo + 63) / 64;
        const int32_t p = lo + lane * step;
        const bool le = p < hi && (int64_t)a.cu[min(p, a.n_seqs)] * g / R + p <= w;
        const int c = __builtin_popcountll(__ballot(le));
        hi = min(hi, lo + c * step);
        lo += (c - 1) * step;
    }
    const int32_t s = __builtin_amdgcn_readfirstlane(lo);
    return make_tile<R>(a, g, s, w - ((int64_t)a.cu[s] * g / R + s), t);
}

// Positions that the row sees: [0, row_limit), 0 for none (at most 2^27: a table holds no more).
__device__ __forceinline__ int32_t row_limit(const Tile &t, int g, int row)
{
    return (int32_t)max(min(t.seen, t.past + row / g + 1), (int64_t)0);
}

// A tile's context is cut into chunks of this many tokens: as near to n_chunks equal parts as multiples
// of `unit` allow.
__device__ __forceinline__ int32_t chunk_of(int32_t lim, int n_chunks, int unit)
{
    const int32_t c = (max(lim, 1) + n_chunks - 1) / n_chunks;
    return (c + unit - 1) / unit * unit;
}

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
// Bound: the cache's bytes, 2*D a token and KV head.  Measured, bf16, 8 query and 2 KV heads of 256: 64
// sequences of 4,096 positions 45.0 us and 8 of 32,768 45.0, 269 MB at 6.0 TB/s (a plain read of that
// size reaches 6.1), the join 4.8 and 5.6 us more; a matrix instruction is busy a tenth of the time.
template <int NT>
constexpr int kRowsOf = NT == 2 ? 8 : 4;
constexpr int kFewWaves = 4;
constexpr int kFewUnit = 128;     // a block of 32 tokens a wave
constexpr int kFewPages = 4096;   // tokens whose pages a wave looks up at once: a 16-token half block a lane

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

// The work is cut by the batch's contexts: chunks of all sequences are about as long as one another, in
// as many as run at once (`budget` for a KV head), so a long context among short ones does not finish
// last.  Sequence s has tiles_s tiles; a tile is cut into n_s chunks, n_s - 1 < seen_s / unit for a unit that
// makes sum_s tiles_s seen_s / unit <= budget.  So there are at most tiles + budget chunks, at most
// `budget` tiles are cut, and those have at most 2 * budget chunks, which get a slot of the workspace each.
struct Cut {
    int32_t s, tile;  // sequence, tile of it
    int32_t slot, n;  // of the tile's first chunk, chunks
};
struct alignas(16) CutList {  // at the workspace's start, for the join
    int32_t n;
    Cut cut[1];
};
constexpr size_t cut_list_bytes(int64_t n) { return 16 + (size_t)n * sizeof(Cut); }

struct FewPlan {
    int32_t budget;            // chunks of a KV head that run at once
    int32_t max_cut, max_slots;  // tiles that may be cut, and chunks of them (none: nothing to join)
};

template <int R>
__device__ __forceinline__ int32_t tiles_of(const Attend &a, int g, int32_t s, bool in)
{
    if (!in) return 0;
    if (!a.cu) return (g + R - 1) / R;
    const int64_t len = min((int64_t)a.cu[s + 1], a.n_tokens) - a.cu[s];
    return (int32_t)((max(len, (int64_t)0) * g + R - 1) / R);
}

__device__ __forceinline__ int32_t seen_of(const Attend &a, int32_t s, bool in)
{
    return in ? (int32_t)min((int64_t)max(a.ctx[s], 0), (int64_t)a.kv.table_width << a.kv.bs_shift) : 0;
}

// Of a tile that sees so many positions (< 2^28, as is the unit).
__device__ __forceinline__ int32_t chunks(int32_t seen, int32_t unit)
{
    return max((int32_t)((uint32_t)(seen + unit - 1) / (uint32_t)unit), 1);
}

struct Sums {  // of a range of sequences: chunks, tiles that are cut, chunks of those
    int32_t all, cut, slots;
    __device__ void add(int32_t tiles, int32_t seen, int32_t unit)
    {
        const int32_t n = chunks(seen, unit);
        all += tiles * n;
        if (n > 1) cut += tiles, slots += tiles * n;
    }
    __device__ Sums scan(int lane) const  // the lanes' up to this one's
    {
        Sums r = *this;
#pragma unroll
        for (int x = 1; x < 64; x *= 2) {
            const Sums o = {__shfl_up(r.all, x), __shfl_up(r.cut, x), __shfl_up(r.slots, x)};
            if (lane >= x) r.all += o.all, r.cut += o.cut, r.slots += o.slots;
        }
        return r;
    }
};

// Chunk w of the call: `z` of tile `c`, whose place in the list of cut tiles is `rank`.
template <int R>
__device__ __forceinline__ bool find_chunk(const Attend &a, int g, int64_t w, int32_t budget, int lane, Cut &c, int32_t &z,
                                           int32_t &rank, int32_t &n_cut)
{
    const int32_t per = (a.n_seqs + 63) / 64;  // sequences of a lane
    const int64_t s0 = (int64_t)lane * per;
    int64_t total = 0;
    int32_t tiles = 0, seen = 0;
    for (int32_t i = 0; i < per; ++i) {
        const bool in = s0 + i < a.n_seqs;
        tiles = tiles_of<R>(a, g, (int32_t)(s0 + i), in);
        seen = seen_of(a, (int32_t)(s0 + i), in);
        total += (int64_t)tiles * seen;
    }
#pragma unroll
    for (int x = 1; x < 64; x *= 2) total += __shfl_xor(total, x);
    const int64_t want = (total + budget - 1) / budget;
    const int32_t unit = (int32_t)max(min((want + kFewUnit - 1) / kFewUnit * kFewUnit, (int64_t)1 << 28), (int64_t)kFewUnit);

    Sums own = {};
    if (per == 1) {
        own.add(tiles, seen, unit);
    } else {
        for (int32_t i = 0; i < per; ++i) {
            const bool in = s0 + i < a.n_seqs;
            own.add(tiles_of<R>(a, g, (int32_t)(s0 + i), in), seen_of(a, (int32_t)(s0 + i), in), unit);
        }
    }
    Sums up = own.scan(lane);
    n_cut = __builtin_amdgcn_readlane(up.cut, 63);
    if (w >= __builtin_amdgcn_readlane(up.all, 63)) return false;
    int at = __builtin_popcountll(__ballot(up.all <= w));  // the lane whose sequences hold it
    Sums base = {__builtin_amdgcn_readlane(up.all - own.all, at), __builtin_amdgcn_readlane(up.cut - own.cut, at),
                 __builtin_amdgcn_readlane(up.slots - own.slots, at)};
    int32_t s = at;
    if (per > 1) {
        const int32_t first = at * per, last = min(first + per, a.n_seqs);
        for (s = first;; s += 64) {  // (ends: the chunk is one of these)
            const bool in = s + lane < last;
            tiles = tiles_of<R>(a, g, s + lane, in);
            seen = seen_of(a, s + lane, in);
            own = {};
            own.add(tiles, seen, unit);
            up = own.scan(lane);
            if (base.all + __builtin_amdgcn_readlane(up.all, 63) > w || s + 64 >= last) break;
            base.all += __builtin_amdgcn_readlane(up.all, 63);
            base.cut += __builtin_amdgcn_readlane(up.cut, 63);
            base.slots += __builtin_amdgcn_readlane(up.slots, 63);
        }
        at = min(__builtin_popcountll(__ballot(base.all + up.all <= w)), 63);
        base.all += __builtin_amdgcn_readlane(up.all - own.all, at);
        base.cut += __builtin_amdgcn_readlane(up.cut - own.cut, at);
        base.slots += __builtin_amdgcn_readlane(up.slots - own.slots, at);
        s += at;
    }
    seen = __builtin_amdgcn_readlane(seen, at);
    c.s = s;
    c.n = chunks(seen, unit);
    const int32_t k = (int32_t)w - base.all;
    c.tile = k / c.n;
    z = k - c.tile * c.n;
    c.slot = base.slots + c.tile * c.n;
    rank = base.cut + c.tile;
    return true;
}

template <int IO>
__device__ __forceinline__ void store_out8(const Attend &a, int64_t off, const float (&y)[8])
{
    store8<IO>(a.out, off, pack8<IO>(y));
}

// Workgroups of a compute unit that the registers let run at once: the accumulators and the block on its
// way grow with D.
constexpr int few_resident(int head_dim) { return head_dim == 256 ? 2 : (head_dim == 128 ? 3 : 4); }

template <int IO, int D, int NT>
__global__ __launch_bounds__(64 * kFewWaves, few_resident(D)) void attend_few_kernel(Attend a, FewPlan p)
{
    constexpr int R = kRowsOf<NT>;
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
    const int32_t lim_last = row_limit(tl, g, tl.row0 + n_rows - 1);  // the most that a row of the tile sees
    const int32_t lim_first = row_limit(tl, g, tl.row0);
    const int32_t chunk = chunk_of((int32_t)tl.seen, cut.n, kFewUnit);  // (a row may end before the last ones)
    const int32_t c0 = (int32_t)min((int64_t)z * chunk, (int64_t)lim_last), c1 = min(c0 + chunk, lim_last);

    // Q: this lane's column is term `t` of row `r`
    const int t = col / R, r = col % R;
    const bool live = t < NT && r < n_rows;
    const int row = tl.row0 + min(r, n_rows - 1);
    const int32_t lim = row_limit(tl, g, row);
    Raw8<IO> qraw[2 * NK];
    {
        const int64_t off = (int64_t)(tl.t0 + row / g) * a.q_tok + (int64_t)(kvh * g + row % g) * a.q_head;
#pragma unroll
        for (int k = 0; k < 2 * NK; ++k) qraw[k] = load8<IO>(a.q, off + (k >> 1) * 64 + grp * 16 + (k & 1) * 8);
    }

    // pages of this wave's half blocks from token `from` on, a lane each
    const int32_t *table = a.kv.tables + tl.s * kv.table_stride;
    int64_t base;
    float ks, vs;
    uint64_t valid_mask;
    auto look_up = [&](int32_t from) {
        base = 0;
        ks = vs = 1.0f;
        bool valid = false;
        const int64_t tok = (int64_t)from + ((lane >> 1) * kFewWaves + wave) * 32 + (lane & 1) * 16;
        if (tok < c1) {
            const int32_t page = table[tok >> kv.bs_shift];
            valid = page >= 0 && page < kv.num_blocks;
            if (valid) {
                ks = kv.k_scale[(int64_t)page * kv.nk + kvh];
                vs = kv.v_scale[(int64_t)page * kv.nk + kvh] * (1.0f / kVUp);
                base = page * kv.c_block;
            }
            base += (tok & (kv.block_size - 1)) * kv.c_tok + kvh * kv.c_head;
        }
        valid_mask = __ballot(valid);
    };
    auto blocks_of = [&](int32_t from) {  // of this wave, in the tokens looked up from there
        const int n = (min(c1 - from, kFewPages) + 31) / 32;
        return n > wave ? (n - wave + kFewWaves - 1) / kFewWaves : 0;
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
    bf16x8 qf[2 * NK];
#pragma unroll
    for (int k = 0; k < 2 * NK; ++k) {
        float x[8];
        unpack8<IO>(qraw[k], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) qf[k][e] = (__bf16)(live ? term<NT>(x[e], t) : 0.0f);
    }

    float m = kNoMax, l = 0.0f;
    f32x4 o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int32_t from = c0;;) {
        for (int it = 0; it < n_mine; ++it) {
            const int32_t tok0 = from + (it * kFewWaves + wave) * 32;
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
            const int32_t mine0 = tok0 + 8 * grp;
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
        if (c1 - from <= kFewPages) break;
        from += kFewPages;
        look_up(from);
        n_mine = blocks_of(from);
        if (n_mine > 0) {
            load_k(0);
            load_v(0);
        }
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
    const bool whole = cut.n == 1;
    Partial<D, R> *part = reinterpret_cast<Partial<D, R> *>(static_cast<char *>(a.workspace) + cut_list_bytes(p.max_cut)) +
                          ((int64_t)(cut.slot + z) * kv.nk + kvh);
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

// ------------------------------------------------------------------ many rows ------------------
// One workgroup: 128 rows (32 a wave) against the context, 64 tokens at a time through LDS.
//
// Both products run in 16 bits (32 x 32 x 16).  S^T = K Q^T: the codes of K are exact in bf16 and fp16, so
// the queries' own type is exact too and fp32 queries take three bf16 terms (each the nearest to what the
// terms before it leave).  K is decoded once, on its way to LDS; its page scale joins the softmax's factor.
// (The 8-bit instruction would take K undecoded, but sums a product's 64 terms with some 13 bits below the
// largest: measured, the scores' sums then were off by 1e-6 of themselves where 32 bits give 4e-8.)
//
// O^T = V^T P^T: V is decoded, its page scale included, on its way to LDS (a code times a power of two is exact
// in bf16), and P taken in bf16 terms: two keep it to 2^-17 for the 16-bit types, as the kernel for few rows
// does, three keep fp32's 2^-24.  One term less would make the errors of the output's rounding visibly larger
// (two e4m3 terms on the 8-bit instruction, 2^-8, took 16 % less time for heads of 256 and raised the error of a
// bf16 output against 64 bits from 0.00165 to 0.00174).
//
// As in the kernel for few rows S^T leaves a lane with the scores of one row, here for 32 of the 64 keys,
// and O^T takes them from there: a step of 16 keys takes 8*a + 4*h + b, a < 2, b < 4, of lane half h.  V goes to
// LDS transposed in that order, a dim's 64 keys in 128 bytes; its 16-byte pieces are swapped by the dim
// (vswap) and 128 bytes left free every D/16 dims, so that the lanes of a read cycle and of a write lie in
// different banks (two other swaps took the same time).  K's rows are 16 bytes longer for the same reason.  V is written a tile later than K, while
// the scores of its own tile are taken, and read in the next: two buffers of each are enough.
//
// Measured: 8 prompts of 4,096 tokens, bf16, 8 query and 2 KV heads of 256: 871 us, 0.63 PFLOP/s (550 GFLOP; with
// the second term of P the matrix instructions do 825, 0.95 PFLOP/s, where a large bf16 product reaches 1.22
// here).  With one wave a SIMD a tile of 64 tokens takes some 7,600 cycles (first and last steps included); the
// matrix unit is busy for 3,100 of them.  Without the softmax's arithmetic it took 807 us, without the
// reads of V 843, without its staging 812, with one term of P 734.  A second wave does not fit (192 registers
// of sums and queries).
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kManyWaves = 4;
constexpr int kManyRows = 32 * kManyWaves;
constexpr int kManyUnit = 64;  // tokens of a tile

// A product in 16 bits: fp16 for fp16 queries, else bf16.
template <int IO>
__device__ __forceinline__ f32x16 mfma16(u32x4 x, u32x4 y, f32x16 c)
{
    if constexpr (IO == kIoF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
}

// Workgroups of a compute unit that run at once.  For D = 256 a wave's sums and queries alone take 192 of
// the 256 registers that two would leave it; for the others they hide one another's waits and
// first and last steps.  Measured: 24 fp16 prompts of up to 900 tokens, D = 128, 176 us with one and 131
// with two; four prompts of 1,500 tokens, D = 64, bf16 47, 42 and 84 us with one, two and three (three
// spill), fp32 57 with one and two; fp32, D = 128, 80 with one and 190 with two (spills).
constexpr int many_resident(int io, int head_dim)
{
    if (head_dim == 256 || (io == kIoF32 && head_dim == 128)) return 1;
    return 2;
}

// The output's sums stay where they are throughout: the compiler otherwise moved all of them from the
// accumulation registers to the others and back in every tile, for the sake of a rescaling that few
// tiles do.  With more than one workgroup it halves the registers between the kinds as soon as any of the
// accumulation registers is named, so there all are of the other kind.
template <int IO, int D>
__device__ __forceinline__ void pin(f32x16 &x)
{
    if constexpr (many_resident(IO, D) == 1) asm volatile("" : "+a"(x));
    else asm volatile("" : "+v"(x));
}

// Eight e4m3 bytes in the 16-bit type (exact). 
template <int IO>
__device__ __forceinline__ u32x4 decode8(uint32_t u, uint32_t v)
{
    if constexpr (IO == kIoF16)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, true))};
    else
        return u32x4{bf16_pair<false>(u, 1.0f), bf16_pair<true>(u, 1.0f), bf16_pair<false>(v, 1.0f), bf16_pair<true>(v, 1.0f)};
}

template <int D>
constexpr int kVB = D / 16;  // dims of V a thread transposes, for four keys

// A sixteen of keys: it has no page; its values may pass 2^90, so P must not exceed 1 beside them (2^8 * 2^90 and
// 2^27 positions still sum below fp32's largest).
constexpr int32_t kNoPage = 1, kLarge = 2;
constexpr int kLargeExp = 80;

template <int D>
struct alignas(16) ManyLds {
    uint8_t k[2][64][2 * D + 16];       // 16-bit keys
    uint8_t v[2][128 * (D + 16)];       // bf16, a dim's 64 keys side by side: see vbyte()
    uint8_t nanv[2][16][D];             // bit b of [w][d]: key 4w + b has a NaN in dim d (written where a row may not see it)
    uint32_t bad[kManyRows][D / 32];    // bit d of a row: it saw a NaN in that dim of V
    int32_t any_bad;
    int32_t nan[2];                     // the last tile in which `nanv` has a bit
    float ks[2][4];                     // by 16 keys: K's scale
    int32_t flags[2][4];                // kNoPage, kLarge
};

// Byte of 16-byte piece `piece` (2 * sixteen of keys + lane half) of dim d.
constexpr int vswap(int d) { return (d & 7) ^ ((d >> 3) & 1); }
template <int D>
__device__ __forceinline__ int vbyte(int d, int piece)
{
    return 128 * (d + d / kVB<D>) + 16 * (piece ^ vswap(d));
}

// The largest of three (of the others where one is NaN), without the canonicalisation that fmaxf costs.
__device__ __forceinline__ float max3(float x, float y, float z)
{
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
    return r;
}

// The larger of a lane's and its counterpart's in the other half of the wave.
__device__ __forceinline__ float max_halves(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max3(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[1]));
}

// Sum over the wave, in every lane.
__device__ __forceinline__ int32_t wave_sum(int32_t x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // row_shr:1, 2, 4, 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // row_bcast:15 and :31
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
    return __builtin_amdgcn_readlane(x, 63);
}

// The tile of the rank-th longest context, and its number w: workgroups start in this order, so that a long
// one does not begin when the others end (4 prompts of 1,500 tokens, bf16, D = 256: 126 us from the batch's last
// tile on, 98 so; 8 of 4,096: 917 and 900).  Tile k of a sequence is ranked by past + floor(R (k + 1) / g); the rank-th
// largest of these is searched for, a sequence a lane.  Batches of more sequences than lanes start from the last
// tile.
template <int R>
__device__ __forceinline__ bool find_long_tile(const Attend &a, int g, int64_t rank, int64_t n_tiles, int lane, Tile &t, int64_t &w)
{
    if (a.n_seqs > 64) {
        w = n_tiles - 1 - rank;
        return find_tile<R>(a, g, w, lane, t);
    }
    const bool in = lane < a.n_seqs;
    const int32_t t0 = !in ? 0 : (a.cu ? a.cu[lane] : lane);
    const int32_t len = !in ? 0 : (a.cu ? (int32_t)max(min((int64_t)a.cu[lane + 1], a.n_tokens) - t0, (int64_t)0) : 1);
    const int32_t tiles = (int32_t)(((int64_t)len * g + R - 1) / R);
    const int32_t past = seen_of(a, lane, in) - len;  // (at most 2^27: a length past the table ranks as the table)
    if (rank >= wave_sum(tiles)) return false;
    auto count = [&](int64_t x) {  // of the lane's tiles that are ranked by x or more: k + 1 >= (x - past) g / R
        const int64_t k1 = ((x - past) * g + R - 1) >> __builtin_ctz(R);
        return tiles - (int32_t)min(max(k1 - 1, (int64_t)0), (int64_t)tiles);
    };
    int32_t lo32 = tiles ? past : 0x7fffffff;
    int32_t span = 0;  // of the ranks, from the least past on (below 2^28: the rows of a call are below 2^26)
#pragma unroll
    for (int x = 1; x < 64; x *= 2) lo32 = min(lo32, __shfl_xor(lo32, x));
    if (tiles) span = (int32_t)min((int64_t)past - lo32 + (int64_t)R * tiles / g + 1, (int64_t)0x7fffffff);
#pragma unroll
    for (int x = 1; x < 64; x *= 2) span = max(span, __shfl_xor(span, x));
    int64_t lo = __builtin_amdgcn_readfirstlane(lo32), hi = lo + __builtin_amdgcn_readfirstlane(span);
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (wave_sum(count(mid)) > rank) lo = mid;
        else hi = mid;
    }
    const int32_t from = count(lo), longer = count(hi), same = from - longer;
    int32_t up = same;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) {
        const int32_t o = __shfl_up(up, x);
        if (lane >= x) up += o;
    }
    const int32_t j = (int32_t)rank - wave_sum(longer);
    const int s = __builtin_popcountll(__ballot(up <= j));
    const int32_t k = __builtin_amdgcn_readlane(tiles - from + j - (up - same), s);
    const int32_t at = __builtin_amdgcn_readlane(t0, s);
    w = (a.cu ? (int64_t)at * g / R + s : (int64_t)s * ((g + R - 1) / R)) + k;
    return make_tile<R>(a, g, s, at, __builtin_amdgcn_readlane(len, s), k, t);
}

template <int IO, int D>
__global__ __launch_bounds__(64 * kManyWaves, many_resident(IO, D)) void attend_many_kernel(Attend a, int n_chunks, int64_t all_tiles)
{
    constexpr int QT = IO == kIoF32 ? 3 : 1;                          // 16-bit terms of Q
    constexpr int N = IO == kIoF32 ? 3 : 2;                           // bf16 terms of P
    constexpr int NS = D / 16, NO = D / 32;
    constexpr int KL = D / 16;             // lanes that load a key row
    constexpr int KR = 64 * kManyWaves / KL, KP = 64 / KR;  // key rows of a pass, passes
    constexpr int VB = kVB<D>;
    const Kv8 &kv = a.kv;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 31, half = lane >> 5;
    // chunks vary fastest: neighbouring workgroups go to the eight dies in turn, and the tiles that are not
    // there (the grid has room for more) come last
    const int z = (int)(blockIdx.x % (unsigned)n_chunks);
    const unsigned unit = blockIdx.x / (unsigned)n_chunks;
    const int g = a.nq / kv.nk, kvh = unit % kv.nk;

    Tile tl;
    int64_t w;
    if (!find_long_tile<kManyRows>(a, g, unit / kv.nk, all_tiles, lane, tl, w)) return;
    const int n_rows = min(kManyRows, tl.rows - tl.row0);
    const int32_t lim_last = row_limit(tl, g, tl.row0 + n_rows - 1);
    const int32_t chunk = chunk_of(lim_last, n_chunks, kManyUnit), c0 = z * chunk;
    if (z > 0 && c0 >= lim_last) return;
    const int32_t c1 = min(c0 + chunk, lim_last);
    const int n_tiles = c1 > c0 ? (c1 - c0 + 63) / 64 : 0;

    __shared__ ManyLds<D> lds;

    // this lane's row, and what the wave's rows see
    const int r = wave * 32 + col;
    const bool live = r < n_rows;
    const int row = tl.row0 + min(r, n_rows - 1);
    const int32_t lim = row_limit(tl, g, row);
    const int32_t wfirst = row_limit(tl, g, tl.row0 + min(wave * 32, n_rows - 1));
    const int32_t wlim = wave * 32 < n_rows ? row_limit(tl, g, tl.row0 + min(wave * 32 + 31, n_rows - 1)) : 0;
    const int32_t first = row_limit(tl, g, tl.row0);  // every row sees the positions before this

    // the scores' factor: its sign goes to Q, and zero makes Q zero, so the largest score is the largest sum
    const float factor = a.scale_log2 != 0.0f ? __builtin_fabsf(a.scale_log2) : 1.0f;
    const float sign = a.scale_log2 < 0.0f ? -1.0f : (a.scale_log2 > 0.0f ? 1.0f : 0.0f);

    // Q: dims 16*s + 8*half .. + 7 of the lane's row
    u32x4 qf[QT][NS];
    {
        const int64_t off = (int64_t)(tl.t0 + row / g) * a.q_tok + (int64_t)(kvh * g + row % g) * a.q_head + half * 8;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            float x[8];
            unpack8<IO>(load8<IO>(a.q, off + s * 16), x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= sign;
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = pack16x2<IO == kIoF16 ? kIoF16 : kIoBF16>(x[2 * i], x[2 * i + 1]);
                    qf[t][s][i] = w;
                    if (t + 1 < QT) {
                        float lo, hi;
                        unpack16x2<kIoBF16>(w, lo, hi);
                        x[2 * i] -= lo;
                        x[2 * i + 1] -= hi;
                    }
                }
        }
    }

    // staging: this thread's pieces of a tile
    const int32_t *table = kv.tables + tl.s * kv.table_stride;
    u32x4 kreg[KP];
    VRow<D> vreg[4];
    const int kr = tid / KL, kc = tid % KL * 16;            // key rows kr, kr + KR, ...
    const int vt = lane & 15, vc = (lane >> 4) + 4 * wave;  // keys 4*vt.., dims VB*vc..
    const int bmask = kv.block_size - 1;                    // tiles begin at multiples of 64: a key's row in its page is its own
    int64_t koff[KP];
#pragma unroll
    for (int p = 0; p < KP; ++p) koff[p] = ((kr + p * KR) & bmask) * kv.c_tok + kc + kvh * kv.c_head;
    const int64_t voff = ((4 * vt) & bmask) * kv.c_tok + vc * VB + kvh * kv.c_head;

    // Pages and scales of 16 tiles, a sixteen of keys a lane; those of the next 16 are fetched on the way.
    struct Lanes {
        int64_t at;   // bytes to the page (a key without one, or past the last tile, reads page 0)
        float ks, vs;
        int32_t flags;
    };
    auto fetch_pages = [&](int group) {
        const int32_t tok = c0 + (group * 64 + lane) * 16;
        int32_t page = -1;
        if (tok < c1) page = table[tok >> kv.bs_shift];
        return page >= 0 && page < kv.num_blocks ? page : -1;
    };
    auto fetch_scales = [&](int32_t page) {
        Lanes x{0, 1.0f, 1.0f, kNoPage};
        if (page >= 0) {
            x.at = page * kv.c_block;
            x.ks = kv.k_scale[(int64_t)page * kv.nk + kvh];
            const int e = scale_exp_of(kv.v_scale[(int64_t)page * kv.nk + kvh]);
            x.vs = pow2(e - kVDown);
            x.flags = e > kLargeExp ? kLarge : 0;
        }
        return x;
    };
    Lanes here{0, 1.0f, 1.0f, kNoPage};
    int32_t page_ahead = -1;
    auto turn_pages = [&](int i) {  // before load_keys(i), in order
        if (i & 7) return;
        if (i & 8) page_ahead = fetch_pages((i >> 4) + 1);
        else here = fetch_scales(i ? page_ahead : fetch_pages(0));
    };
    auto page_at = [&](int l) {
        const uint32_t lo = __shfl((int)(uint32_t)here.at, l), hi = __shfl((int)(uint32_t)((uint64_t)here.at >> 32), l);
        return (int64_t)(((uint64_t)hi << 32) | lo);
    };
    float ks_lane = 1.0f;  // of the keys loaded last, where this lane holds one of the tile's sixteens
    int32_t flags_lane = kNoPage, info = -1;
    const uint8_t *pv = kv.v;  // this thread's rows of the same tile's V, their scale (0: no page)
    float vs_next = 0.0f, vs = 0.0f;
    auto load_keys = [&](int i) {
        const int at = (i & 15) * 4;
        const uint8_t *pk[KP];
#pragma unroll
        for (int p = 0; p < KP; ++p) pk[p] = kv.k + page_at(at + ((kr + p * KR) >> 4)) + koff[p];
#pragma unroll
        for (int p = 0; p < KP; ++p) kreg[p] = *reinterpret_cast<const u32x4 *>(pk[p]);
        pv = kv.v + page_at(at + (vt >> 2)) + voff;
        vs_next = __shfl(here.flags & kNoPage ? 0.0f : here.vs, at + (vt >> 2));
        info = lane - at;
        ks_lane = here.ks;
        flags_lane = here.flags;
    };
    auto load_values = [&]() {  // of the tile whose keys were loaded last
        vs = vs_next;
#pragma unroll
        for (int j = 0; j < 4; ++j) vreg[j] = load_vrow<D>(pv + j * kv.c_tok);
    };
    auto store_info = [&](int i) {
        if ((unsigned)info < 4u) {  // every wave writes the same
            lds.ks[i & 1][info] = ks_lane;
            lds.flags[i & 1][info] = flags_lane;
        }
    };
    // What no row sees may hold anything: it must not reach the product; and where some rows see a NaN and
    // others do not, the product goes on without it and the rows are told.
    auto clean_v = [&](int i) {
        const int32_t t0 = c0 + i * 64;
        if (t0 + 64 <= first && !__any(vs == 0.0f)) return;  // (the lanes' keys are all of the tile's)
        bool nan = false;
#pragma unroll
        for (int w = 0; w < VB / 4; ++w) {
            uint32_t bits = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t y = vreg[j].w[w];
                asm volatile("" : "+v"(y));  // not before the branch
                if (vs == 0.0f || t0 + 4 * vt + j >= lim_last) y = 0;
                const uint32_t n = (((y & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;  // 1 in a NaN's byte
                bits |= n << j;
                vreg[j].w[w] = y & ~(n * 0xffu);
            }
            *reinterpret_cast<uint32_t *>(&lds.nanv[i & 1][vt][vc * VB + 4 * w]) = bits;
            nan |= bits != 0;
        }
        if (nan) lds.nan[i & 1] = i;
    };
    // keys 4*vt..: sixteen vt/4, lane half vt%2, first or second half of the piece; dims VB*vc..
    const int vput = 128 * (VB + 1) * vc + 16 * ((vt >> 2) * 2 + (vt & 1)) + 8 * ((vt >> 1) & 1);
    constexpr int kSlices = KP + VB / 4;
    auto store_slice = [&](int n, int i) {  // of tile i's V and tile i + 1's keys
        if (n < KP) {
            uint8_t *kb = &lds.k[(i + 1) & 1][kr][2 * kc] + n * KR * (2 * D + 16);
            const u32x4 x = kreg[n < KP ? n : 0];
            *reinterpret_cast<u32x4 *>(kb) = decode8<IO>(x[0], x[1]);
            *reinterpret_cast<u32x4 *>(kb + 16) = decode8<IO>(x[2], x[3]);
            return;
        }
        // the bytes of two keys side by side, then bf16 pairs (key, key + 1) of one dim
        const int w = n - KP;
        const uint32_t r0 = vreg[0].w[w], r1 = vreg[1].w[w], r2 = vreg[2].w[w], r3 = vreg[3].w[w];
        const uint32_t a0 = __builtin_amdgcn_perm(r1, r0, 0x05010400u), a1 = __builtin_amdgcn_perm(r3, r2, 0x05010400u);
        const uint32_t b0 = __builtin_amdgcn_perm(r1, r0, 0x07030602u), b1 = __builtin_amdgcn_perm(r3, r2, 0x07030602u);
        auto put = [&](int e, uint32_t x, uint32_t y) {
            const int j = 4 * w + e;  // of the thread's dims
            *reinterpret_cast<uint2 *>(lds.v[i & 1] + ((vput ^ (16 * (vswap(j) ^ vswap(VB * vc)))) + 128 * j)) = make_uint2(x, y);
        };
        put(0, bf16_pair<false>(a0, vs), bf16_pair<false>(a1, vs));
        put(1, bf16_pair<true>(a0, vs), bf16_pair<true>(a1, vs));
        put(2, bf16_pair<false>(b0, vs), bf16_pair<false>(b1, vs));
        put(3, bf16_pair<true>(b0, vs), bf16_pair<true>(b1, vs));
    };

    float m = kNoMax, l = 0.0f;
    f32x16 o[NO];
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q) o[i][q] = 0.0f;
#pragma unroll
    for (int i = 0; i < NO; ++i) pin<IO, D>(o[i]);

    // P of the tile before, in terms: its product with V is taken while the next softmax runs
    u32x4 pf[N][4];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) pf[n][j] = u32x4{0, 0, 0, 0};
    // Step u of the product with V: dims 64 * (u / 4).., the sixteen u % 4 of keys; the sums of two pieces of
    // dims take turns, so neighbouring instructions do not depend on one another.
    constexpr int kSteps = 2 * NO;
    int vget[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) vget[j] = vbyte<D>(col, 2 * j + half);
    auto value_piece = [&](int i, int u, int e) {
        return *reinterpret_cast<const u32x4 *>(lds.v[i & 1] + vget[u & 3] + (4096 + 4096 / VB) * (2 * (u >> 2) + e));
    };
    auto value_product = [&](int u, u32x4 x0, u32x4 x1) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            o[2 * (u >> 2)] = mfma16<kIoBF16>(x0, pf[n][u & 3], o[2 * (u >> 2)]);
            o[2 * (u >> 2) + 1] = mfma16<kIoBF16>(x1, pf[n][u & 3], o[2 * (u >> 2) + 1]);
        }
    };
    // The dims in which this lane's row sees a NaN in tile i's V, half of them a lane (rare).
    auto mark_nan = [&](int i) {
        if (lds.nan[i & 1] != i) return;
        const int32_t seen = lim - (c0 + i * 64);
#pragma unroll 1
        for (int d = half * (D / 2); d < (half + 1) * (D / 2); ++d) {
            uint32_t bad_d = 0;
#pragma unroll 1
            for (int w = 0; w < 16; ++w) bad_d |= lds.nanv[i & 1][w][d] & ((1u << min(max(seen - 4 * w, 0), 4)) - 1);
            if (bad_d) {
                lds.bad[r][d >> 5] |= 1u << (d & 31);
                lds.any_bad = 1;
            }
        }
    };

    if (tid < 2) lds.nan[tid] = -2;
    if (tid == 2) lds.any_bad = 0;
    for (int i = tid; i < kManyRows * NO; i += 64 * kManyWaves) lds.bad[i / NO][i % NO] = 0;
    for (int i = tid; i < 8 * (D + 16); i += 64 * kManyWaves)  // before the first tile: nothing
        reinterpret_cast<u32x4 *>(lds.v[1])[i] = u32x4{0, 0, 0, 0};
    if (n_tiles > 0) {
        turn_pages(0);
        load_keys(0);
        load_values();
        store_info(0);
#pragma unroll
        for (int n = 0; n < KP; ++n) store_slice(n, -1);
        load_keys(1);
    }
    // tiles that this wave's rows see, then those that it only helps to stage
    const int n_mine = min(n_tiles, wlim > c0 ? (wlim - c0 + 63) / 64 : 0);
    int it = 0;
    for (; it < n_mine; ++it) {
        const int32_t t0 = c0 + it * 64;
        // K of tile `it` and V of tile it - 1 are in LDS; K of tile it - 1 and V of tile it - 2 have been read
        __syncthreads();
        clean_v(it);
        store_info(it + 1);
        turn_pages(it + 2);
        __builtin_amdgcn_sched_barrier(0);

        // The scores, step by step, their operands read kAhead steps before their use; beside them the
        // tile's V and the next tile's K go to LDS, and those after them are asked for.  (Past the last tile
        // both are done for nobody.)
        constexpr int kAhead = many_resident(IO, D) > 1 ? 2 : 4;
        const uint8_t *kb = &lds.k[it & 1][col][16 * half];
        auto key_piece = [&](int k, int h) { return *reinterpret_cast<const u32x4 *>(kb + h * 32 * (2 * D + 16) + k * 32); };
        f32x16 s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 16; ++q) s[h][q] = 0.0f;
        u32x4 piece[kAhead][2];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            piece[k][0] = key_piece(k, 0);
            piece[k][1] = key_piece(k, 1);
        }
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            constexpr int kPer = (kSlices + NS / 2 - 1) / (NS / 2);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int n = 0; n < QT; ++n) s[h] = mfma16<IO>(piece[k % kAhead][h], qf[n][k], s[h]);
                if (k + kAhead < NS) piece[k % kAhead][h] = key_piece(k + kAhead, h);
            }
#pragma unroll
            for (int n = k * kPer; n < (k + 1) * kPer; ++n)
                if (n < kSlices) store_slice(n, it);
            if (k == NS / 2) {
                load_values();
                load_keys(it + 2);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        float f[4];  // by 16 keys: the scores' factor
        int32_t flags[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = lds.ks[it & 1][j];
            flags[j] = lds.flags[it & 1][j];
        }
        constexpr int kVAhead = many_resident(IO, D) > 1 ? 1 : 2;
        u32x4 vx[kVAhead + 1][2];  // V's operands
#pragma unroll
        for (int u = 0; u < kVAhead; ++u) {
            vx[u][0] = value_piece(it - 1, u, 0);
            vx[u][1] = value_piece(it - 1, u, 1);
        }

        // register 4a + b of s[h]: key 32h + 8a + 4*half + b
        if (t0 + 64 > wfirst || __any((flags[0] | flags[1] | flags[2] | flags[3]) & kNoPage)) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int key = 32 * h + 8 * (q >> 2) + 4 * half + (q & 3);
                    if (t0 + key >= lim || (flags[2 * h + (q >> 3)] & kNoPage)) s[h][q] = -__builtin_inff();
                }
        }
        __builtin_amdgcn_sched_barrier(0);
        // The softmax, and between its steps the tile before's product with V.
        float top[4], m_new = m, ladd = 0.0f;
        bool moves = false;
        u32x4 pn[N][4];
        auto begin = [&]() {
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // the largest score of each sixteen
                const int h = j >> 1, q = 8 * (j & 1);
                f[j] = fmaxf(f[j] * factor, 0x1p-126f);  // not 0, which would make a masked -infinity NaN
                top[j] = max3(max3(max3(s[h][q], s[h][q + 1], s[h][q + 2]), s[h][q + 3], s[h][q + 4]), s[h][q + 5], s[h][q + 6]);
                top[j] = max3(top[j], s[h][q + 7], s[h][q + 7]) * f[j];
            }
            // the maximum moves only where it has grown by 2^8: until then p exceeds 1 and nothing is lost (but
            // beside large values, where the sums have no room for it, it moves at once)
            const float m_top = max_halves(max3(max3(top[0], top[1], top[2]), top[3], m));
            const bool large = (flags[0] | flags[1] | flags[2] | flags[3]) & kLarge;
            moves = __any(m_top > m + (large ? 0.0f : 8.0f));
            m_new = moves ? m_top : m;
        };
        auto two = [&](int n) {  // p of registers 2*(n%8).. of s[n/8]: two keys of sixteen n/4
            float p[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) p[q] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n >> 3][2 * (n & 7) + q], f[n >> 2], -m_new));
            ladd += p[0] + p[1];
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const uint32_t w = pack16x2<kIoBF16>(p[0], p[1]);
                float lo, hi;
                unpack16x2<kIoBF16>(w, lo, hi);
                p[0] -= lo;
                p[1] -= hi;
                pn[t][n >> 2][n & 3] = w;
            }
        };
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            if (u + kVAhead < kSteps) {
                vx[(u + kVAhead) % (kVAhead + 1)][0] = value_piece(it - 1, u + kVAhead, 0);
                vx[(u + kVAhead) % (kVAhead + 1)][1] = value_piece(it - 1, u + kVAhead, 1);
            }
            value_product(u, vx[u % (kVAhead + 1)][0], vx[u % (kVAhead + 1)][1]);
            if (u == 0) begin();
#pragma unroll
            for (int n = 0; n < 16; ++n)
                if (u > 0 && n * (kSteps - 1) / 16 == u - 1) two(n);
            __builtin_amdgcn_sched_barrier(0);
        }
        // (P is finished here and not beyond the branch below, where nothing runs beside it)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(pn[n][j]));
        asm volatile("" : "+v"(ladd));
        __builtin_amdgcn_sched_barrier(0);
        if (moves) {
            const float c = __builtin_amdgcn_exp2f(m - m_new);
            l *= c;
#pragma unroll
            for (int i = 0; i < NO; ++i) {
                pin<IO, D>(o[i]);  // nor read before the branch
                o[i] *= c;
                pin<IO, D>(o[i]);
            }
            m = m_new;
        }
        l += ladd;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) pf[n][j] = pn[n][j];
#pragma unroll
        for (int i = 0; i < NO; ++i) pin<IO, D>(o[i]);
        mark_nan(it - 1);
    }
    for (const int last = it; it <= n_tiles; ++it) {
        __syncthreads();
        if (it < n_tiles) {
            clean_v(it);
            store_info(it + 1);
            turn_pages(it + 2);
#pragma unroll
            for (int n = 0; n < kSlices; ++n) store_slice(n, it);
            load_values();
            load_keys(it + 2);
        }
        if (it == last) {
#pragma unroll
            for (int u = 0; u < kSteps; ++u) value_product(u, value_piece(it - 1, u, 0), value_piece(it - 1, u, 1));
            mark_nan(it - 1);
        }
    }

    l += __shfl_xor(l, 32);
    if (!live) return;
    if (lds.any_bad) {
#pragma unroll
        for (int i = 0; i < NO; ++i) {
            const uint32_t b = lds.bad[r][i] >> (4 * half);  // both halves of a row's dims are marked by lanes of this wave
#pragma unroll
            for (int q = 0; q < 16; ++q)
                if ((b >> (8 * (q >> 2) + (q & 3))) & 1) o[i][q] = __builtin_nanf("");
        }
    }
    const int64_t tok = tl.t0 + row / g;
    const int head = kvh * g + row % g;
    if (lim_last <= chunk) {
        const float inv = out_factor(l);  // (a row that saw nothing has summed nothing)
#pragma unroll
        for (int i = 0; i < NO; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) y[b] = o[i][4 * e + b] * inv;
                const int64_t at = tok * a.o_tok + head * a.o_head + 32 * i + 8 * e + 4 * half;
                if constexpr (IO == kIoF32)
                    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
                else
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
                        make_uint2(pack16x2<IO>(y[0], y[1]), pack16x2<IO>(y[2], y[3]));
            }
        if (a.lse && half == 0)
            a.lse[tok * a.nq + head] = l == 0.0f ? -__builtin_inff() : 0.69314718055994531f * (m + __log2f(l));
    } else {
        Partial<D, kManyRows> *part = static_cast<Partial<D, kManyRows> *>(a.workspace) +
                                      ((w * kv.nk + kvh) * n_chunks + z);
#pragma unroll
        for (int i = 0; i < NO; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<float4 *>(&part->o[r][32 * i + 8 * e + 4 * half]) =
                    make_float4(o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]);
        if (half == 0) {
            part->ml[r][0] = m;
            part->ml[r][1] = l;
        }
    }
}

// Joins a tile's chunks: some waves a row, D/4 lanes over its dims and the rest over the chunks.  The
// largest maximum is found first, so the chunks' parts add up without waiting for one another.  A row of many
// chunks takes the eight waves of a workgroup, one of few chunks two (64 rows in 40 chunks: 6.0 us with
// eight and 9.1 with two; 2 prompts of 300 tokens in six: 21.6 and 9.4).
constexpr int kJoinThreads = 512, kJoinMany = 16;

template <int IO, int D, int R, int ROWS>  // rows of a workgroup
__global__ __launch_bounds__(kJoinThreads) void attend_join_kernel(Attend a, int n_chunks, int32_t max_cut)
{
    constexpr int kThreads = kJoinThreads / ROWS, kWaves = kThreads / 64;  // of a row
    constexpr int LANES = D / 4, PARTS = kThreads / LANES, U = 4;
    const int g = a.nq / a.kv.nk, kvh = blockIdx.y, lane = threadIdx.x & 63;
    const int mine = threadIdx.x / kThreads, tid = threadIdx.x % kThreads, rr = blockIdx.z * ROWS + mine;
    Tile tl;
    int n;
    const Partial<D, R> *part;
    int64_t stride = 1;  // from a chunk's part to the next one's
    if constexpr (R == kManyRows) {
        if (!find_tile<R>(a, g, blockIdx.x, lane, tl)) return;
        const int32_t lim_last = row_limit(tl, g, min(tl.row0 + R, tl.rows) - 1);
        const int32_t chunk = chunk_of(lim_last, n_chunks, kManyUnit);
        if (lim_last <= chunk) return;
        n = (int)((lim_last + chunk - 1) / chunk);
        part = static_cast<const Partial<D, R> *>(a.workspace) + ((int64_t)blockIdx.x * a.kv.nk + kvh) * n_chunks;
    } else {
        const CutList *list = static_cast<const CutList *>(a.workspace);
        if ((int64_t)blockIdx.x >= list->n) return;
        const Cut c = list->cut[blockIdx.x];
        make_tile<R>(a, g, c.s, c.tile, tl);
        n = c.n;
        part = reinterpret_cast<const Partial<D, R> *>(static_cast<const char *>(a.workspace) + cut_list_bytes(max_cut)) +
               ((int64_t)c.slot * a.kv.nk + kvh);
        stride = a.kv.nk;
    }
    const bool live = rr < min(R, tl.rows - tl.row0);
    if (!live) n = 0;
    const int d = tid % LANES * 4, sub = tid / LANES;

    __shared__ float sm[ROWS][kWaves], sl[ROWS][PARTS];
    __shared__ f32x4 sy[ROWS][PARTS][LANES];
    float m = kNoMax;
    for (int z = tid; z < n; z += kThreads) m = fmaxf(m, part[z * stride].ml[rr][0]);
#pragma unroll
    for (int x = 1; x < 64; x *= 2) m = fmaxf(m, __shfl_xor(m, x));
    if (lane == 0) sm[mine][tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sm[mine][w]);

    float l = 0.0f;
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int z0 = sub; z0 < n; z0 += U * PARTS) {
        f32x4 po[U];
        float f[U], pl[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Partial<D, R> &p = part[min(z0 + u * PARTS, n - 1) * stride];
            f[u] = p.ml[rr][0];
            pl[u] = p.ml[rr][1];
            po[u] = *reinterpret_cast<const f32x4 *>(&p.o[rr][d]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (z0 + u * PARTS >= n) break;
            const float e = __builtin_amdgcn_exp2f(f[u] - m);
            l += pl[u] * e;
            y += po[u] * e;
        }
    }
    sy[mine][sub][d / 4] = y;
    if (d == 0) sl[mine][sub] = l;
    __syncthreads();
    const int e = tid;
    if (!live || e >= D / 8) return;
    float ll = 0.0f, r[8] = {};
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        ll += sl[mine][p];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] += sy[mine][p][2 * e + (i >> 2)][i & 3];
    }
    const int rw = tl.row0 + rr;
    const int64_t tok = tl.t0 + rw / g;
    const int head = kvh * g + rw % g;
    const float inv = out_factor(ll);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = ll == 0.0f ? 0.0f : r[i] * inv;
    store_out8<IO>(a, tok * a.o_tok + head * a.o_head + 8 * e, r);
    if (a.lse && e == 0)
        a.lse[tok * a.nq + head] = ll == 0.0f ? -__builtin_inff() : 0.69314718055994531f * (m + __log2f(ll));
}

// ------------------------------------------------------------------ launchers ------------------
struct Plan {
    bool many;
    int64_t tiles;
    int rows;         // of a tile
    int64_t grid;     // few rows: chunks at most
    FewPlan few;
    int n_chunks;     // many rows: of a tile
    size_t bytes;     // of the workspace
};

// Tiles of many rows where a sequence's rows of a KV head would fill more than four tiles of few rows, which
// read the cache once each.  Measured (us, few against many; bf16, 8 query and 2 KV heads of 256): 3
// sequences with 20,000 tokens behind them, 16 rows each 30 / 43, 32 rows 40 / 43, 48 rows 79 / 46; 16
// sequences with 1,500, 32 rows 28 / 32, 48 rows 44 / 33.  fp32 (4 rows a tile): 16 rows 43 / 66, 24 rows 90 / 68.
// The host does not see lengths: the rule takes the call's average, and a call that mixes prompts with
// single tokens has one kernel for both (one prompt of 2,048 tokens and seven tokens at 100,000 positions:
// 4.2 ms together, 0.09 and 0.14 in calls of their own; one of 4,096 and a thousand at 500: 0.64, and 0.21 and 0.15).
constexpr int64_t kFewTiles = 4;
Plan make_plan(int64_t n_tokens, int32_t n_seqs, int32_t nq, int32_t nk, int32_t head_dim, int io, bool one_token,
               int32_t table_width, int32_t block_size)
{
    Plan p{};
    const int64_t g = nq / nk, cap = std::max<int64_t>(1, (int64_t)table_width * block_size);
    const int few_rows = io == kIoF32 ? kRowsOf<3> : kRowsOf<2>;
    p.many = n_tokens * g > kFewTiles * few_rows * n_seqs;
    p.rows = p.many ? kManyRows : few_rows;
    p.tiles = one_token ? (int64_t)n_seqs * ((g + p.rows - 1) / p.rows) : n_tokens * g / p.rows + n_seqs;
    const int64_t unit = p.many ? kManyUnit : kFewUnit, most = (cap + unit - 1) / unit;
    const size_t part = (size_t)(p.rows * (head_dim + 2) * 4) * nk;
    if (p.many) {
        // The context is cut where the tiles are fewer than the compute units; twice as many chunks took 63 us
        // where these take 48 (3 sequences of 16 tokens behind 20,011, bf16, D = 256), and two a compute unit,
        // which D = 128 and 64 have room for, 37 and 30 us for 33 and 26 (2 of 300 behind 500).
        // (Of the tiles in the grid those are counted that sequences of equal lengths would have.)
        const int64_t fill = 256, seq_rows = (n_tokens * g + n_seqs - 1) / n_seqs;
        const int64_t likely = std::min(p.tiles, n_seqs * ((seq_rows + p.rows - 1) / p.rows));
        p.n_chunks = (int)std::min(most, std::max<int64_t>(1, fill / (likely * nk)));
        if (p.n_chunks > 1) p.bytes = part * (size_t)(p.tiles * p.n_chunks);
        return p;
    }
    p.few.budget = std::max(1, 256 * few_resident(head_dim) / nk);
    p.grid = std::min(p.tiles + p.few.budget, p.tiles * most);
    if (most > 1) {
        p.few.max_cut = (int32_t)std::min<int64_t>(p.tiles, p.few.budget);
        p.few.max_slots = (int32_t)std::min<int64_t>(2 * p.few.budget, p.tiles * most);
        p.bytes = cut_list_bytes(p.few.max_cut) + part * (size_t)p.few.max_slots;
    }
    return p;
}

template <int IO, int D>
hipError_t launch_attend_d(const Attend &a, hipStream_t stream)
{
    constexpr int NT = IO == kIoF32 ? 3 : 2;
    const Plan p = make_plan(a.n_tokens, a.n_seqs, a.nq, a.kv.nk, D, IO, a.cu == nullptr, a.kv.table_width, a.kv.block_size);
    const int32_t nk = a.kv.nk, g = a.nq / nk;
    if (p.many) {
        const dim3 grid((unsigned)(p.tiles * nk * p.n_chunks));
        attend_many_kernel<IO, D><<<grid, 64 * kManyWaves, 0, stream>>>(a, p.n_chunks, p.tiles);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || p.n_chunks == 1) return e;
        const unsigned tiles = (unsigned)p.tiles;
        if (p.n_chunks > kJoinMany)
            attend_join_kernel<IO, D, kManyRows, 1><<<dim3(tiles, nk, kManyRows), kJoinThreads, 0, stream>>>(a, p.n_chunks, 0);
        else
            attend_join_kernel<IO, D, kManyRows, 4><<<dim3(tiles, nk, kManyRows / 4), kJoinThreads, 0, stream>>>(a, p.n_chunks, 0);
    } else {
        attend_few_kernel<IO, D, NT><<<dim3((unsigned)p.grid, nk), 64 * kFewWaves, 0, stream>>>(a, p.few);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || p.few.max_cut == 0) return e;
        const int rows = a.cu ? p.rows : std::min(p.rows, g);
        const dim3 join((unsigned)p.few.max_cut, nk, rows);
        attend_join_kernel<IO, D, kRowsOf<NT>, 1><<<join, kJoinThreads, 0, stream>>>(a, 0, p.few.max_cut);
    }
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
    return make_plan(n_tokens, n_seqs, nq, nk, head_dim, io, one_token, table_width, block_size).bytes;
}

hipError_t launch_attend(const Attend &a, int io, hipStream_t stream)
{
    if (io == kIoBF16) return launch_attend_io<kIoBF16>(a, stream);
    if (io == kIoF16) return launch_attend_io<kIoF16>(a, stream);
    return launch_attend_io<kIoF32>(a, stream);
}

}  // namespace mrope
