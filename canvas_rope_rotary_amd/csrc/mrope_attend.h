// What the attention kernels over the 8-bit paged cache share: the work of a workgroup (tiles of rows, chunks of
// contexts), decoding, the parts of a tile's chunks and the kernel that joins them.
#pragma once

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

constexpr int kFewWaves = 4;
constexpr int kFewUnit = 128;     // a block of 32 tokens a wave
constexpr int kFewPages = 4096;   // tokens whose pages a wave looks up at once: a 16-token half block a lane

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

// The largest of three (of the others where one is NaN): one instruction, without the canonicalisation that fmaxf costs, and
// one that the compiler knows to read a matrix instruction's result, which needs wait states.
__device__ __forceinline__ float max3(float x, float y, float z)
{
    return __builtin_elementwise_maximumnum(__builtin_elementwise_maximumnum(x, y), z);
}

// The larger of a lane's and its counterpart's in the other half of the wave.
__device__ __forceinline__ float max_halves(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max3(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[1]));
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

constexpr int kManyWaves = 4;
constexpr int kManyRows = 32 * kManyWaves;
constexpr int kManyUnit = 64;  // tokens of a tile

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

}  // namespace
}  // namespace mrope
