// Attention of trees of drafted tokens over the 8-bit paged K/V cache (mrope_attend_tree_kv8).
//
//   out[t, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q[t, h] . k_j - max),
//
// over the positions j that query token i (of len) of a sequence of ctx positions sees: those before ctx - len,
// and ctx - len + b for the bits b that are set in its row of the mask.  Tiles, chunks of contexts and the join are those of
// mrope_attend.h; a row is a (token, head of the group) pair, row = i * g + head.
//
// One workgroup: 32 or 64 rows against a chunk of the context, eight waves (four for fp32 heads of 256), two a SIMD, that
// take 32 tokens each in turn with thirty-two rows, or all 64 where the registers hold them (heads of up to 128).
// S^T = K Q^T (32 x 32 x 16): a lane ends with the scores of one row of each thirty-two (its column) for sixteen of the
// tokens, keys 8a + 4h + b, a, b < 4, of lane half h; O^T = V^T P^T takes sixteen tokens a step and each lane's operand is
// what it has there, if V's comes in the same order.  So nothing moves between lanes but for the maximum, and the parts of
// waves with other tokens meet only once, at the end.  Codes are exact in 16 bits, V with its scale.  P is taken in two bf16
// terms for the 16-bit types (2^-17, as the other kernels over this cache do) and three for fp32, fp32 queries in three (each
// the bf16 nearest to what the terms before it leave).
//
// Codes come to LDS by loads that pass no register, a block ahead: into a ring of the wave's own, so no wave waits for
// another, or into one that two waves with other rows share, so a block is brought once for 64 rows.  The queries wait in
// LDS in the order of the instruction's operand.
//
// Only blocks that reach past ctx - len, or into a page that is not there, look at the mask.
//
// Measured, heads of 256 in bf16, 8 of 2 KV heads (a call, and the medians of its kernels under a trace): 64 trees of 32 tokens
// at 4,096 positions 119 to 121 us (128 + 4.9 for a join with nothing to join), 103 GFLOP with P's second term, 0.87 PFLOP/s; 8 trees
// of 16 at 32,000 positions 73 to 79 us (79 + 6.8), 263 MB of codes, 3.3 to 3.6 TB/s.  The matrix instructions are busy for
// 45 % of a wave's cycles (99,000 of 221,000; of the latter's 33 %) and the others, decoding and the softmax, issue for about as
// many, few of them at the same time: scores, softmax and product of a block follow one another, in both waves of a SIMD.  That
// is the order they are written in and no limit of the hardware: in a loop of one 32 x 32 x 16 instruction and three conversions
// two waves take 19.0 ns a step, where the two kinds alone take 14.7 and 14.1.  fp32, three terms of both (207 GFLOP for the 64 trees):
// 214 us, 0.97 PFLOP/s, heads of 128 110, of 64 65.  A call of one tree at a short context is a chain of
// waits, 12 us: 2 to find the chunk, 3 for the page's number, then its codes and scales, 1 for the queries, 2 for a block,
// 4 for the parts to meet, most of them for code that comes for the first time.
#include <algorithm>

#include "mrope_attend.h"

namespace mrope {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int IO>
constexpr int kQTerms = IO == kIoF32 ? 3 : 1;
template <int IO>
constexpr int kPTerms = IO == kIoF32 ? 3 : 2;

template <int IO>
__device__ __forceinline__ f32x16 mfma_scores(u32x4 x, u32x4 y, f32x16 c)
{
    if constexpr (IO == kIoF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 mfma_bf16(u32x4 x, u32x4 y, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
}

// Two e4m3 bytes of a key as the scores' 16-bit type (exact).  bf16 takes the page's scale at once; fp16 has no
// room for it, and the scores are multiplied instead.
template <int IO, bool HI>
__device__ __forceinline__ uint32_t key_pair(uint32_t u, float scale)
{
    if constexpr (IO == kIoF16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, HI));
    else return bf16_pair<HI>(u, scale);
}

// Workgroups of a compute unit that run at once: registers hold two waves a SIMD but for 32 rows of 64 dims.
constexpr int tree_resident(int io, int head_dim, int nb) { return head_dim == 64 && io != kIoF32 && nb == 1 ? 2 : 1; }

// Running sum over the lanes: within sixteens, then a sixteen's last to those behind it.
__device__ __forceinline__ int32_t running(int32_t x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
    return x;
}

// The largest of the lanes' (none of them negative).
__device__ __forceinline__ int32_t largest(int32_t x)
{
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));
    return __builtin_amdgcn_readlane(x, 63);
}

// The work of workgroup `id`: a chunk of a tile, of chunks that are as long as one another and fit those that run at once:
// at most `budget` a KV head, or the tiles, none of them cut.  A chunk is `unit` times U tokens: the least that fits, which
// lies between the sum's share and, as a tile adds less than one chunk to its share, that of what the tiles leave of the budget
// (more than 64 sequences, a second look at each for each trial, take the latter).  Tiles stay whole where the cut does not
// shorten the longest by GAIN tokens, times the share of the budget that it takes, since parts are written and read again (16
// trees of 32 at 1,000 positions, heads of 256: 26.3 us whole, 30.0 in two; 64 of 16 at 4,096 in tiles of 64 rows: 97.3 and
// 80.3).  `z` is the chunk's place in its tile,
// `rank` that of the tile in the list of cut ones.  The chunks of all heads in order, an eighth to each XCD (id % 8): tiles of
// the same context and heads of the same pages meet in its L2.
template <int R, int U, int GAIN>
__device__ __forceinline__ bool find_fit(const AttendTree &a, int g, int32_t id, int32_t budget, int lane, Cut &c, int32_t &z,
                                         int32_t &rank, int32_t &n_cut, int32_t &kvh, Tile &t)
{
    int32_t t0, len, ctx, seen, tiles, units;
    auto read = [&](int32_t s) {
        const int32_t at = min(s, a.n_seqs - 1), next = a.cu[at + 1], c_at = a.ctx[at];
        t0 = a.cu[at];
        len = s < a.n_seqs ? (int32_t)min((int64_t)next, a.n_tokens) - t0 : 0;
        ctx = max(c_at, 0);
        seen = (int32_t)min((int64_t)ctx, (int64_t)a.kv.table_width << a.kv.bs_shift);  // (at most 2^27)
        tiles = (int32_t)(((int64_t)max(len, 0) * g + R - 1) / R);
        units = (seen + U - 1) / U;
    };
    int32_t all = 0, total = 0, longest = 0;
    for (int32_t s = lane; s - lane < a.n_seqs; s += 64) {
        read(s);
        all += tiles;
        longest = max(longest, tiles ? units : 0);
        total += tiles * units;  // (matters where the tiles are fewer than the budget, and is below 2^31 then)
    }
    all = __builtin_amdgcn_readlane(running(all), 63);
    total = __builtin_amdgcn_readlane(running(total), 63);
    const int32_t left = budget - all;
    auto chunks_here = [&](int32_t unit) { return max((int32_t)((uint32_t)(units + unit - 1) / (uint32_t)unit), 1); };
    auto count_of = [&](int32_t unit) {
        int32_t c = 0;
        for (int32_t s = lane; s - lane < a.n_seqs; s += 64) {
            if (a.n_seqs > 64) read(s);
            c += tiles * chunks_here(unit);
        }
        return (int32_t)__builtin_amdgcn_readlane(running(c), 63);
    };
    int32_t unit = 1 << 30, count = all;  // of chunks
    if (left > 0) {
        unit = max((int32_t)(((uint32_t)total + left - 1) / (uint32_t)left), 1);
        for (int32_t lo = max((int32_t)(((uint32_t)total + budget - 1) / (uint32_t)budget), 1); a.n_seqs <= 64 && lo < unit;) {
            const int32_t mid = (lo + unit) >> 1;
            if (count_of(mid) <= budget) unit = mid;
            else lo = mid + 1;
        }
        count = count_of(unit);
        const int32_t cut = largest(max(longest - unit, 0)) * U;  // (at most 2^27)
        if ((int64_t)cut * budget < (int64_t)GAIN * count) unit = 1 << 30, count = all;
    }
    const int32_t nk = a.kv.nk, share = (int32_t)(((int64_t)count * nk + 7) / 8), v = id % 8 * share + id / 8;
    const bool mine = id / 8 < share && v < count * nk;
    if (!mine && id) return false;
    const int32_t w = mine ? v / nk : 1 << 30;
    kvh = v % nk;

    Sums base = {0, 0, 0};
    bool found = false;
    for (int32_t s0 = 0; s0 < a.n_seqs; s0 += 64) {
        if (a.n_seqs > 64) read(s0 + lane);
        const int32_t n = chunks_here(unit);
        const int32_t own = tiles * n, own_cut = n > 1 ? tiles : 0;
        const int32_t up = running(own), up_cut = running(own_cut), up_slots = running(n > 1 ? own : 0);
        if (!found && base.all + __builtin_amdgcn_readlane(up, 63) > w) {
            found = true;
            const int at = min(__builtin_popcountll(__ballot(base.all + up <= w)), 63);
            c.s = s0 + at;
            c.n = __builtin_amdgcn_readlane(n, at);
            const int32_t k = w - base.all - __builtin_amdgcn_readlane(up - own, at);
            c.tile = k / c.n;
            z = k - c.tile * c.n;
            c.slot = base.slots + __builtin_amdgcn_readlane(up_slots - (n > 1 ? own : 0), at) + c.tile * c.n;
            rank = base.cut + __builtin_amdgcn_readlane(up_cut - own_cut, at) + c.tile;
            t.s = c.s;
            t.t0 = __builtin_amdgcn_readlane(t0, at);
            t.rows = __builtin_amdgcn_readlane(len, at) * g;
            t.row0 = c.tile * R;
            t.seen = __builtin_amdgcn_readlane(seen, at);
            t.past = (int64_t)__builtin_amdgcn_readlane(ctx, at) - __builtin_amdgcn_readlane(len, at);
            if (id) break;  // (the first workgroup goes on, for the sum)
        }
        base.all += __builtin_amdgcn_readlane(up, 63);
        base.cut += __builtin_amdgcn_readlane(up_cut, 63);
        base.slots += __builtin_amdgcn_readlane(up_slots, 63);
    }
    n_cut = base.cut;
    return found;
}

// Codes of 32 tokens on their way, as they lie in the cache but for the order of a row's 16-byte pieces (K) and of the
// rows (V): so chosen that the lanes of a read lie in different banks.
template <int D>
struct alignas(16) Block {
    uint8_t k[32 * D], v[32 * D];
};

// A workgroup: WAVES waves, GROUPS groups of which take other rows of the same tokens; a wave has 32 * NB rows.
template <int IO, int D, int NB, int GROUPS, int WAVES>
struct alignas(16) TreeLds {
    static constexpr int kShares = WAVES / GROUPS;                // waves with the same rows
    static constexpr int kBuffers = GROUPS > 1 ? 2 : 1;
    static constexpr int kSlice = kShares > 4 && D == 256 ? 16 : 32;  // rows whose parts meet at a time: as LDS has room
    union {
        struct {
            Block<D> ring[kShares][kBuffers];                     // blocks of the waves with the same tokens
            u32x4 q[NB * GROUPS][kQTerms<IO>][D / 16][64];    // the operand's pieces by lane
        };
        struct {                                                  // when the last block is done
            float o[kShares][kSlice][D + 4];
            float ml[kShares][32 * NB * GROUPS][2];
        };
    };
};

// 16 bytes a lane from global memory (g, the same in all lanes, and an offset) to LDS, where the lanes' lie one after
// the other from `l` on.  (A buffer load: for the global form the compiler waits at the next use of LDS for all of it.)
__device__ __forceinline__ void to_lds16(const uint8_t *g, uint32_t off, uint8_t *l)
{
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(g), 0, -1, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)l, 16, off, 0, 0, 0);
}

// Where row r of 32 has its 16-byte piece p of K, and its row of V.
template <int D>
__device__ __forceinline__ int key_piece_of(int r, int p)
{
    if constexpr (D == 256) return p ^ (r & 15);
    else if constexpr (D == 128) return p ^ ((r >> 1) & 7);
    else return p ^ ((r >> 2) & 3);
}
template <int D>
__device__ __forceinline__ int value_row_of(int r)
{
    return D == 256 ? r : r ^ ((r >> 2) & 1);
}

// The bytes of V that a lane holds of a token: D / 32 dims.
template <int D>
struct VPiece {
    uint32_t w[D == 256 ? 2 : 1];
};
#define MROPE_LDS __attribute__((address_space(3)))
template <int D>
__device__ __forceinline__ VPiece<D> load_vpiece(const uint8_t *p)
{
    VPiece<D> r;
    if constexpr (D == 256) {
        const uint64_t x = *reinterpret_cast<const uint64_t *>(p);
        r.w[0] = (uint32_t)x, r.w[1] = (uint32_t)(x >> 32);
    } else if constexpr (D == 128) {
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
        r.w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
    return r;
}
// From LDS (as such: a read that only the optimiser knows to be one waits for every load to LDS on its way).
template <int D>
__device__ __forceinline__ VPiece<D> read_vpiece(const uint8_t *p)
{
    VPiece<D> r;
    if constexpr (D == 256) {
        const uint64_t x = *(const MROPE_LDS uint64_t *)p;
        r.w[0] = (uint32_t)x, r.w[1] = (uint32_t)(x >> 32);
    } else if constexpr (D == 128) {
        r.w[0] = *(const MROPE_LDS uint32_t *)p;
    } else {
        r.w[0] = *(const MROPE_LDS uint16_t *)p;
    }
    return r;
}
#undef MROPE_LDS

// V's page scale (2^8 smaller) beside which the running maximum follows at once.
constexpr float kLargeScale = 0x1p72f;

template <int IO, int D, int NB, int GROUPS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, tree_resident(IO, D, NB) * WAVES / 4) void attend_tree_kernel(AttendTree a, FewPlan p)
{
    constexpr int R = 32 * NB * GROUPS, QT = kQTerms<IO>, N = kPTerms<IO>, kShares = WAVES / GROUPS;
    constexpr int NS = D / 16;   // steps of a score
    constexpr int NO = D / 32;   // dims of V that a lane holds of a token, and 32-dim tiles of O^T
    const Kv8 &kv = a.kv;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int col = lane & 31, half = lane >> 5;
    const int share = wave % kShares, row0 = wave / kShares * 32 * NB;  // the wave's tokens, its first row of the tile
    const int g = a.nq / kv.nk;

    Cut cut;
    Tile tl;
    int32_t z, rank, n_cut, kvh;
    const bool found = find_fit<R, 32 * kShares, (D == 256 ? 768 : 1536) * tree_resident(IO, D, NB)>(a, g, blockIdx.x, p.budget, lane, cut, z, rank, n_cut, kvh, tl);
    CutList *list = static_cast<CutList *>(a.workspace);
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.max_cut) list->n = min(n_cut, p.max_cut);
    if (!found) return;
    if (cut.n > 1) {
        if (rank >= p.max_cut || cut.slot + cut.n > p.max_slots) return;  // (not for offsets that grow)
        if (z == 0 && kvh == 0 && threadIdx.x == 0) list->cut[rank] = cut;
    }
    const int n_rows = min(R, tl.rows - tl.row0);
    const int32_t len = tl.rows / g;
    const int32_t seen = __builtin_amdgcn_readfirstlane((int32_t)tl.seen);
    const int32_t past = __builtin_amdgcn_readfirstlane((int32_t)tl.past);  // (>= -2^31: ctx >= 0)
    const int32_t open = min(max(past, 0), seen);                     // every row sees the positions before this
    const int32_t chunk = chunk_of(seen, cut.n, 32 * kShares);
    const int32_t c0 = __builtin_amdgcn_readfirstlane((int32_t)min((int64_t)z * chunk, (int64_t)seen));
    const int32_t c1 = __builtin_amdgcn_readfirstlane(min(c0 + chunk, seen));

    __shared__ TreeLds<IO, D, NB, GROUPS, WAVES> lds;

    // Blocks of 32 tokens: this wave's i-th begins at c0 + (i kShares + share) * 32.  Pages of 32 of them at a time, those
    // of a sixteen of tokens a lane.
    const int32_t *table = kv.tables + tl.s * kv.table_stride;
    int32_t tok_lane, page_lane;
    int64_t base;
    float ks_lane, vs_lane;
    bool valid;
    uint64_t valid_mask;
    auto ask_pages = [&](int i) {
        tok_lane = c0 + ((i + (lane >> 1)) * kShares + share) * 32 + (lane & 1) * 16;  // (at most 2^27 + 2^13)
        page_lane = table[min(tok_lane, c1 - 1) >> kv.bs_shift];
    };
    auto use_pages = [&] {
        valid = tok_lane < c1 && page_lane >= 0 && page_lane < kv.num_blocks;
        const int64_t page = valid ? page_lane : 0;
        ks_lane = kv.k_scale[page * kv.nk + kvh];
        vs_lane = kv.v_scale[page * kv.nk + kvh];
        base = page * kv.c_block + (tok_lane & (kv.block_size - 1)) * kv.c_tok + kvh * kv.c_head;
        valid_mask = __ballot(valid);
    };
    auto settle = [&] {
        ks_lane = valid ? ks_lane : 1.0f;
        vs_lane = valid ? pow2(scale_exp_of(vs_lane) - kVDown) : 1.0f;  // (finite, whatever nobody sees)
        asm volatile("" : "+v"(ks_lane), "+v"(vs_lane));  // (they have come: no later wait is for them)
    };
    struct Info {  // of a block: scales and whether the page is there, by sixteens of tokens
        float ks0, ks1, vs0, vs1;
        bool ok0, ok1;
    };
    constexpr bool kTogether = GROUPS > 1;  // waves with other rows of the same tokens share a block
    Block<D> *ring = lds.ring[share];
    // An instruction brings 1 KB: RI rows, and the lanes' places within them.
    constexpr int RI = 1024 / D, NI = 32 / RI, PR = D / 16;
    constexpr int KV = 16 / RI < NI ? 16 / RI : NI;  // places that differ: K's order of pieces goes by a row of sixteen
    uint32_t koff[KV], voff[1];
#pragma unroll
    for (int i = 0; i < KV; ++i) koff[i] = (lane / PR) * (uint32_t)kv.c_tok + 16 * key_piece_of<D>(i * RI + lane / PR, lane % PR);
    voff[0] = value_row_of<D>(lane / PR) * (uint32_t)kv.c_tok + 16 * (lane % PR);
    auto fetch = [&](int i, const uint8_t *cache, const auto &off, uint8_t *to) {
        constexpr int kPeriod = sizeof(off) / 4;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int at = 2 * (i & 31) + u;
            const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)base, at);
            const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)base >> 32), at);
            const int64_t b = (int64_t)(((uint64_t)hi << 32) | lo);
#pragma unroll
            for (int j = u * NI / 2; j < (u + 1) * NI / 2; ++j)
                to_lds16(cache + (b + (j * RI) % 16 * kv.c_tok), off[j % kPeriod], to + 1024 * j);
        }
    };
    auto info = [&](int i) {
        const int at = 2 * (i & 31);
        Info x;
        x.ks0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ks_lane), at));
        x.ks1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ks_lane), at + 1));
        x.vs0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(vs_lane), at));
        x.vs1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(vs_lane), at + 1));
        x.ok0 = (valid_mask >> at) & 1, x.ok1 = (valid_mask >> (at + 1)) & 1;
        return x;
    };
    auto fetch_keys = [&](int i) { fetch(i, kv.k, koff, ring[kTogether ? i & 1 : 0].k); };
    auto fetch_values = [&](int i) { fetch(i, kv.v, voff, ring[kTogether ? i & 1 : 0].v); };
    auto fetch_mine = [&](int i) {  // of two groups the first brings keys, the other values
        if (wave < kShares) fetch_keys(i);
        else fetch_values(i);
    };
    auto look_up = [&](int i) {
        ask_pages(i);
        use_pages();
        settle();
    };
    const int n_all = (c1 - c0 + 31) / 32, n_mine = n_all > share ? (n_all - share + kShares - 1) / kShares : 0;
    if (n_mine > 0) ask_pages(0);

    // The queries (past the last row: that one again) are asked for while the pages' numbers are on their way.
    constexpr int kQLoads = (NS + WAVES - 1) / WAVES;
    decltype(load8<IO>(a.q, 0)) raw[NB * GROUPS][kQLoads];
#pragma unroll
    for (int nb = 0; nb < NB * GROUPS; ++nb) {
        const int row = tl.row0 + min(nb * 32 + col, n_rows - 1);
        const int64_t off = (int64_t)(tl.t0 + row / g) * a.q_tok + (int64_t)(kvh * g + row % g) * a.q_head + 16 * half;
#pragma unroll
        for (int i = 0; i < kQLoads; ++i) {
            const int s = (i * WAVES + wave) % NS;
            raw[nb][i] = load8<IO>(a.q, off + 32 * (s >> 1) + 8 * (s & 1));
        }
    }
    Info next{};
    if (n_mine > 0) {
        use_pages();
        if constexpr (kTogether) {
            fetch_mine(0);
        } else {
            fetch_keys(0);
            fetch_values(0);
        }
        settle();
        next = info(0);
    }

    // the scores' factor: its sign goes to Q, and zero makes Q zero, so the largest score is the largest sum
    const float factor = a.scale_log2 != 0.0f ? __builtin_fabsf(a.scale_log2) : 1.0f;
    const float sign = a.scale_log2 < 0.0f ? -1.0f : (a.scale_log2 > 0.0f ? 1.0f : 0.0f);

    // The queries: piece s of lane (col, half) is dims 32 * (s / 2) + 16 * half + 8 * (s % 2) .. + 7 of row col.
#pragma unroll
    for (int nb = 0; nb < NB * GROUPS; ++nb)
#pragma unroll
        for (int i = 0; i < kQLoads; ++i) {
            float x[8];
            unpack8<IO>(raw[nb][i], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= sign;
            u32x4 w[QT];
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[t][e] = pack16x2<IO == kIoF16 ? kIoF16 : kIoBF16>(x[2 * e], x[2 * e + 1]);
                    if (t + 1 < QT) {
                        float lo, hi;
                        unpack16x2<kIoBF16>(w[t][e], lo, hi);
                        x[2 * e] -= lo;
                        x[2 * e + 1] -= hi;
                    }
                }
#pragma unroll
            for (int t = 0; t < QT; ++t) lds.q[nb][t][(i * WAVES + wave) % NS][lane] = w[t];  // (by two waves the same, of few pieces)
        }
    __syncthreads();

    int32_t itok[NB];  // the query token of this lane's row of each thirty-two
#pragma unroll
    for (int n = 0; n < NB; ++n) itok[n] = (tl.row0 + min(row0 + n * 32 + col, n_rows - 1)) / g;
    // Which of the tokens tok0 .. + 31 query token i sees: bit q for tok0 + q.
    auto sees = [&](int32_t i, int32_t tok0, bool ok0, bool ok1) {
        const int32_t j = tok0 - past;  // (the tree's token at tok0)
        const uint64_t *row = a.mask + (int64_t)(tl.t0 + i) * a.mask_words;
        const int32_t w = j >> 6;
        auto word = [&](int32_t k) { return k < 0 ? ~0ull : (k < a.mask_words ? row[k] : 0ull); };
        uint64_t bits = word(w) >> (j & 63);
        if ((j & 63) > 32) bits |= word(w + 1) << (64 - (j & 63));
        const int32_t n = min(min(len - j, seen - tok0), 32);
        const uint32_t there = (ok0 ? 0xffffu : 0u) | (ok1 ? 0xffff0000u : 0u);
        return n > 0 ? (uint32_t)bits & (0xffffffffu >> (32 - n)) & there : 0u;
    };

    float m[NB], l[NB];
    f32x16 o[NB][NO];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        m[n] = kNoMax;
        l[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < NO; ++i) {
#pragma unroll
            for (int q = 0; q < 16; ++q) o[n][i][q] = 0.0f;
        }
    }

    uint32_t nan = 0;    // a block with a mask had one in V
    u32x4 pf[NB][2][N];  // P's terms by step of sixteen tokens
    Info now{};          // of the block that the wave is at
    bool edge = false;   // it has a mask (wave-uniform)

    // Block `it`: its scores and their softmax.
    auto scores = [&](int it, bool more) {
        const int32_t tok0 = c0 + (it * kShares + share) * 32;
        const Block<D> &blk = ring[kTogether ? it & 1 : 0];
        now = next;
        const float kscale = col < 16 ? now.ks0 : now.ks1;
        int here = lane;  // (opaque: the queries stay in LDS and are read anew)
        asm volatile("" : "+v"(here));

        // The scores, step by step, their operands read some steps before their use.
        constexpr int kSteps = NS * NB * QT, kAhead = 4 < kSteps ? 4 : kSteps, kKeysAhead = 3 < NS / 2 ? 3 : NS / 2;
        u32x4 kp[kKeysAhead], q[kAhead];
        const u32x4 *queries = &lds.q[wave / kShares * NB][0][0][0];
        auto query = [&](int i) { return queries[((i % NB * QT + i / NB % QT) * NS + i / (NB * QT)) * 64 + here]; };
        auto key_piece = [&](int k) { return *reinterpret_cast<const u32x4 *>(blk.k + col * D + 16 * key_piece_of<D>(col, 2 * k + half)); };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) q[i] = query(i);
        // its keys have come (its values, NI instructions, may be on their way)
        if constexpr (!kTogether) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NI) : "memory");
        else if (more) {
            if ((it + 1) % 32 == 0) look_up(it + 1);
            fetch_mine(it + 1);
            next = info(it + 1);
        }
#pragma unroll
        for (int k = 0; k < kKeysAhead; ++k) kp[k] = key_piece(k);
        f32x16 s[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[n][e] = 0.0f;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            const u32x4 x = kp[(k >> 1) % kKeysAhead];
            const int h = k & 1;
            const u32x4 f = {key_pair<IO, false>(x[2 * h], kscale), key_pair<IO, true>(x[2 * h], kscale),
                             key_pair<IO, false>(x[2 * h + 1], kscale), key_pair<IO, true>(x[2 * h + 1], kscale)};
            if (h && (k >> 1) + kKeysAhead < NS / 2) kp[(k >> 1) % kKeysAhead] = key_piece((k >> 1) + kKeysAhead);
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const int i = (k * QT + t) * NB + n;
                    s[n] = mfma_scores<IO>(f, q[i % kAhead], s[n]);
                    if (i + kAhead < kSteps) q[i % kAhead] = query(i + kAhead);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!kTogether && more) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the keys have been read
            if ((it + 1) % 32 == 0) look_up(it + 1);
            fetch_keys(it + 1);
            next = info(it + 1);
        }

        edge = tok0 + 32 > open || !now.ok0 || !now.ok1;
        // (fp16: not 0, which would make a masked -infinity NaN, nor past fp32)
        const float f0 = IO == kIoF16 ? fminf(fmaxf(now.ks0 * factor, 0x1p-126f), 0x1p127f) : factor;
        const float f1 = IO == kIoF16 ? fminf(fmaxf(now.ks1 * factor, 0x1p-126f), 0x1p127f) : factor;
        // the maximum moves only where it has grown by 2^8: until then p exceeds 1 and nothing is lost (but
        // beside large values, where the sums have no room for it, it moves at once)
        const float lag = fmaxf(now.vs0, now.vs1) >= kLargeScale ? 0.0f : 8.0f;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            if (edge) {
                const uint32_t vis = sees(itok[n], tok0, now.ok0, now.ok1) >> (4 * half);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (!(vis >> (8 * (e >> 2) + (e & 3)) & 1)) s[n][e] = -__builtin_inff();
            }
            auto top8 = [&](int e) {
                return max3(max3(s[n][e], s[n][e + 1], s[n][e + 2]), max3(s[n][e + 3], s[n][e + 4], s[n][e + 5]), max3(s[n][e + 6], s[n][e + 7], s[n][e + 7]));
            };
            const float t0 = top8(0) * f0, t1 = top8(8) * f1;
            const float top = max_halves(max3(t0, t1, t1));
            if (__any(top > m[n] + lag)) {
                const float m_new = fmaxf(m[n], top);
                const float c = __builtin_amdgcn_exp2f(m[n] - m_new);
                l[n] *= c;
#pragma unroll
                for (int i = 0; i < NO; ++i) o[n][i] *= c;
                m[n] = m_new;
            }
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][e], e < 8 ? f0 : f1, -m[n]));
                float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][e + 1], e < 8 ? f0 : f1, -m[n]));
                l[n] += p0 + p1;
#pragma unroll
                for (int t = 0; t < N; ++t) {
                    const uint32_t w = pack16x2<kIoBF16>(p0, p1);
                    pf[n][e >> 3][t][(e & 7) >> 1] = w;
                    if (t + 1 < N) {
                        float lo, hi;
                        unpack16x2<kIoBF16>(w, lo, hi);
                        p0 -= lo;
                        p1 -= hi;
                    }
                }
            }
        }

    };

    // Then its product with V.
    auto product = [&](int it, bool more) {
        const Block<D> &blk = ring[kTogether ? it & 1 : 0];
        if constexpr (!kTogether) {  // its values have come (the next block's keys may be on their way)
            if (more) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NI) : "memory");
            else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        // V's bytes: step u of sixteen tokens, tokens 16 u + 8 a + 4 half + b
        VPiece<D> vp[2][8];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                vp[u][j] = read_vpiece<D>(blk.v + value_row_of<D>(16 * u + 8 * (j >> 2) + 4 * half + (j & 3)) * D + col * NO);
        // A NaN that some rows see and others do not, or that nobody sees, must not reach the product: the product
        // goes on without it, and the rows that see it are told at the end.
        if (edge) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int w = 0; w < (D == 256 ? 2 : 1); ++w) {
                        uint32_t &x = vp[u][j].w[w];
                        const uint32_t bad = (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;  // 1 in a NaN's byte
                        nan |= bad;
                        x &= ~(bad * 0xffu);
                    }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float vscale = u ? now.vs1 : now.vs0;
#pragma unroll
            for (int w = 0; w < (NO + 3) / 4; ++w) {
                // bytes of two tokens side by side, then bf16 pairs (token, next token) of one dim
                uint32_t lo[4], hi[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    lo[j] = __builtin_amdgcn_perm(vp[u][2 * j + 1].w[w], vp[u][2 * j].w[w], 0x05010400u);
                    if (NO > 2) hi[j] = __builtin_amdgcn_perm(vp[u][2 * j + 1].w[w], vp[u][2 * j].w[w], 0x07030602u);
                }
#pragma unroll
                for (int e = 0; e < (NO < 4 ? NO : 4); ++e) {
                    u32x4 fv;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t b = e < 2 ? lo[j] : hi[j];
                        fv[j] = e & 1 ? bf16_pair<true>(b, vscale) : bf16_pair<false>(b, vscale);
                    }
#pragma unroll
                    for (int t = 0; t < N; ++t)
#pragma unroll
                        for (int n = 0; n < NB; ++n) o[n][4 * w + e] = mfma_bf16(fv, pf[n][u][t], o[n][4 * w + e]);
                }
            }
            if (!kTogether && u == 1 && more) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the values have been read
                fetch_values(it + 1);
            }
        }
    };

    if constexpr (!kTogether) {
        for (int it = 0; it < n_mine; ++it) {
            scores(it, it + 1 < n_mine);
            product(it, it + 1 < n_mine);
        }
    } else {
        // The first group brings a block's keys, the second its values, while the block before is at work, to where the one
        // before that was: its readers have passed the barrier since.  (A barrier that leaves codes on their way, as
        // __syncthreads does not.)
        static_assert(GROUPS == 2, "two groups share a block");
        for (int it = 0; it < (n_all + kShares - 1) / kShares; ++it) {
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");  // what was asked for has come, what was read too
            if (it < n_mine) {
                scores(it, it + 1 < n_mine);
                product(it, it + 1 < n_mine);
            }
        }
    }

    if (__any(nan != 0)) {  // (rare) the blocks with a mask again: the rows that see a NaN have it in these dims
#pragma unroll 1
        for (int it = 0; it < n_mine; ++it) {
            const int32_t tok0 = c0 + (it * kShares + share) * 32;
            if ((it & 31) == 0) look_up(it);
            const int at = 2 * (it & 31);
            const bool ok0 = (valid_mask >> at) & 1, ok1 = (valid_mask >> (at + 1)) & 1;
            if (tok0 + 32 <= open && ok0 && ok1) continue;
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
                const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)base, at + u);
                const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)base >> 32), at + u);
                const int64_t b = (int64_t)(((uint64_t)hi << 32) | lo);
                VPiece<D> vp[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) vp[j] = load_vpiece<D>(kv.v + b + (8 * (j >> 2) + 4 * half + (j & 3)) * kv.c_tok + col * NO);
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const uint32_t vis = sees(itok[n], tok0, ok0, ok1) >> (16 * u + 4 * half);
                    u32x4 mine;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mine[j] = (vis >> (8 * (j >> 1) + 2 * (j & 1)) & 1 ? 0x3f80u : 0u) | (vis >> (8 * (j >> 1) + 2 * (j & 1) + 1) & 1 ? 0x3f800000u : 0u);
#pragma unroll
                    for (int i = 0; i < NO; ++i) {
                        u32x4 ind;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t x = vp[2 * j].w[i / 4] >> (8 * (i % 4)), y = vp[2 * j + 1].w[i / 4] >> (8 * (i % 4));
                            ind[j] = ((x & 0x7f) == 0x7f ? 0x3f80u : 0u) | ((y & 0x7f) == 0x7f ? 0x3f800000u : 0u);
                        }
                        f32x16 cnt;
#pragma unroll
                        for (int e = 0; e < 16; ++e) cnt[e] = 0.0f;
                        cnt = mfma_bf16(ind, mine, cnt);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (cnt[e] > 0.0f) o[n][i][e] = __builtin_nanf("");
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
        }
    }

    // the parts of the waves with the same rows meet in LDS, some rows at a time
    __syncthreads();  // (the ring and the queries have been read)
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        l[n] += __shfl_xor(l[n], 32);
        if (half == 0) {
            lds.ml[share][row0 + n * 32 + col][0] = m[n];
            lds.ml[share][row0 + n * 32 + col][1] = l[n];
        }
    }
    const bool whole = cut.n == 1;
    Partial<D, R> *part = reinterpret_cast<Partial<D, R> *>(static_cast<char *>(a.workspace) + cut_list_bytes(p.max_cut)) +
                          ((int64_t)(cut.slot + z) * kv.nk + kvh);
    constexpr int kSlice = TreeLds<IO, D, NB, GROUPS, WAVES>::kSlice, kSlices = 32 / kSlice;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll 1
    for (int w = 0; w < kSlices * GROUPS; ++w) {  // (rolled: what runs once is bound by the fetch of its code)
        const int slice = w % kSlices, first = (w / kSlices * NB + n) * 32 + slice * kSlice;
        if (first >= n_rows) continue;
        if (n || w) __syncthreads();  // the rows before have been read
        if (wave / kShares == w / kSlices && col / kSlice == slice) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float *dst = &lds.o[share][col % kSlice][(8 * (e >> 2) + 4 * half + (e & 3)) * NO];
                if constexpr (NO >= 4) {
#pragma unroll
                    for (int i = 0; i < NO; i += 4) *reinterpret_cast<f32x4 *>(dst + i) = f32x4{o[n][i][e], o[n][i + 1][e], o[n][i + 2][e], o[n][i + 3][e]};
                } else {
#pragma unroll
                    for (int i = 0; i < NO; ++i) dst[i] = o[n][i][e];
                }
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < min(kSlice, n_rows - first) * (D / 8); e += 64 * WAVES) {
            const int r = e / (D / 8), rr = first + r, d = e % (D / 8) * 8;
            float mm = kNoMax, ll = 0.0f, y[8] = {};
#pragma unroll
            for (int i = 0; i < kShares; ++i) mm = fmaxf(mm, lds.ml[i][rr][0]);
#pragma unroll
            for (int i = 0; i < kShares; ++i) {
                const float f = __builtin_amdgcn_exp2f(lds.ml[i][rr][0] - mm);
                ll += lds.ml[i][rr][1] * f;
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] += lds.o[i][r][d + j] * f;
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
    bool wide;      // tiles of 64 rows, else of 32
    int64_t tiles, grid;
    FewPlan few;
    size_t bytes;   // of the workspace
};

struct Shape {
    int nb, groups, waves;  // (see the kernel)
    constexpr int rows() const { return 32 * nb * groups; }
    constexpr int unit() const { return 32 * waves / groups; }  // a chunk's tokens are a multiple of
};

// fp32 queries take three times the room in LDS: tiles of 32 rows, and of 256 dims four waves.  64 rows of 256 dims are two
// waves' (a wave's registers hold 32), of fewer dims one wave's: for 128 dims 70.9 us against two waves' 81.9 (64 trees of
// 32 at 4,096 positions), for 64 54.6 and 84.0.
constexpr Shape shape_of(int io, int head_dim, bool wide)
{
    if (io == kIoF32) return {1, 1, head_dim == 256 ? 4 : 8};
    if (!wide) return {1, 1, 8};
    return head_dim == 256 ? Shape{1, 2, 8} : Shape{2, 1, 8};
}

TreePlan make_plan(int64_t n_tokens, int32_t n_seqs, int32_t nq, int32_t nk, int32_t head_dim, int io, int32_t table_width,
                   int32_t block_size)
{
    TreePlan p{};
    const int64_t g = nq / nk, cap = std::max<int64_t>(1, (int64_t)table_width * block_size);
    const int64_t seq_rows = (n_tokens * g + n_seqs - 1) / n_seqs;
    // Tiles of 64 rows decode a block for twice the rows, tiles of 32 spread further: narrow as long as all of them run at once
    // (us, narrow and wide.  Fewer: 3 trees of 250 at 2,047 positions 41.7 and 51.0, 64 of 16 at 4,096 80.4 and 83.3, in heads of
    // 128 27.9 and 38.8, 47.5 and 52.3, of 64 22.5 and 29.9, 32.9 and 39.2.  More: 64 of 32 at 4,096 136.3 and 126.0, 256 of 16 at
    // 1,000 116.5 and 91.9, in heads of 128 83.1 and 73.4, 75.3 and 61.5, of 64 50.1 and 47.6, but 41.7 and 45.0).
    p.wide = n_seqs * ((seq_rows + 31) / 32) * nk > 256 && io != kIoF32;
    const Shape shape = shape_of(io, head_dim, p.wide);
    const int64_t rows = shape.rows(), most = (cap + shape.unit() - 1) / shape.unit();
    p.tiles = n_tokens * g / rows + n_seqs;
    p.few.budget = std::max(1, 256 * tree_resident(io, head_dim, shape.nb) / nk);
    p.grid = std::min(std::max<int64_t>(p.tiles, p.few.budget), p.tiles * most);
    if (most > 1) {
        p.few.max_cut = (int32_t)std::min<int64_t>(p.tiles, p.few.budget);
        p.few.max_slots = (int32_t)std::min<int64_t>(p.few.budget, p.tiles * most);
        p.bytes = cut_list_bytes(p.few.max_cut) + (size_t)(rows * (head_dim + 2) * 4) * nk * (size_t)p.few.max_slots;
    }
    return p;
}

template <int IO, int D, bool WIDE>
hipError_t launch_tree_shape(const AttendTree &a, const TreePlan &p, hipStream_t stream)
{
    constexpr Shape S = shape_of(IO, D, WIDE);
    const unsigned grid = (unsigned)((p.grid * a.kv.nk + 7) / 8 * 8);  // as many for each XCD
    attend_tree_kernel<IO, D, S.nb, S.groups, S.waves><<<grid, 64 * S.waves, 0, stream>>>(a, p.few);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.few.max_cut == 0) return e;
    // Waves a row of the join by the chunks a tile may have (us, eight and two waves: one tree of 8 at 30,000 positions 29.0
    // and 43.2, two of 16 at 16,000 29.5 and 36.8; 8 of 16 at 32,000 80.5 and 79.4, 16 of 16 at 8,000 55.9 and 50.8).
    const unsigned tiles = (unsigned)p.few.max_cut;
    if (p.few.max_slots > kJoinMany * p.few.max_cut)
        attend_join_kernel<IO, D, S.rows(), 1><<<dim3(tiles, a.kv.nk, S.rows()), kJoinThreads, 0, stream>>>(a, 0, p.few.max_cut);
    else
        attend_join_kernel<IO, D, S.rows(), 4><<<dim3(tiles, a.kv.nk, S.rows() / 4), kJoinThreads, 0, stream>>>(a, 0, p.few.max_cut);
    return hipGetLastError();
}

template <int IO, int D>
hipError_t launch_tree_d(const AttendTree &a, hipStream_t stream)
{
    const TreePlan p = make_plan(a.n_tokens, a.n_seqs, a.nq, a.kv.nk, D, IO, a.kv.table_width, a.kv.block_size);
    if constexpr (IO != kIoF32) {
        if (p.wide) return launch_tree_shape<IO, D, true>(a, p, stream);
    }
    return launch_tree_shape<IO, D, false>(a, p, stream);
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

size_t attend_tree_workspace_bytes(int64_t n_tokens, int32_t n_seqs, int32_t nq, int32_t nk, int32_t head_dim, int io,
                                   int32_t table_width, int32_t block_size)
{
    return make_plan(n_tokens, n_seqs, nq, nk, head_dim, io, table_width, block_size).bytes;
}

hipError_t launch_attend_tree(const AttendTree &a, int io, hipStream_t stream)
{
    if (io == kIoBF16) return launch_tree_io<kIoBF16>(a, stream);
    if (io == kIoF16) return launch_tree_io<kIoF16>(a, stream);
    return launch_tree_io<kIoF32>(a, stream);
}

}  // namespace mrope
