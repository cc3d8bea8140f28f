// Verification of drafted tokens against the target's probabilities (mrope_verify_tree).
//
// The walk begins at token 0 of a sequence.  At token a, with r = p_a, c = 0 and Z = 1, the children of a are
// tested in order: child x is accepted if u_x * q_a(x) * Z < r(x) (q = 1 where the drafts were not drawn) and the walk
// goes on from it; else c += Z, r = max(p_a - c q_a, 0), Z = sum r (drafts that were not drawn: r(x) = 0 and
// Z = max(Z - r(x), 0)).  (Refusals one after the other take max(max(p - Z1 q, 0) - Z2 q, 0) = max(p - (Z1 + Z2) q, 0)
// of the row, so one number holds them.)  Where no child is left the next token is drawn from r: the first
// whose running sum passes u_next times the sum of r.  All in 64 bits; the order of the sums is fixed.
//
// Only rows that have to be are read whole: the one where a walk ends, and drawn trees' rows whose first
// child is refused and has siblings.  Such a sum separates the walk before it from the walk after it, so a launch
// ("round") continues each sequence's walk as far as it goes without a new sum and then adds its row up, cut into
// parts over workgroups.  Every workgroup of a sequence does the walk for itself (tests of single elements, fetched
// side by side for all tokens), so nothing waits for another workgroup.  The last launch finds the part and the
// element; walks that the rounds did not end it ends by itself, one workgroup a sequence.
// Bound: where sequences are few, latency (tokens, their probabilities, the walk, the row: 7.2 us for a round of one chain of
// six over 248,094 ids, 3.7 for the last launch; 64 trees of 32 in bf16 16.6 and 4.7 for 32 MB); where they are many, for
// fp32 the reads (500 rows: 496 MB in 92 us, 5.4 TB/s, and 6 for the last launch), for the 16-bit types nothing alone: 2,000 rows
// of fp16 or bf16 take 237 and 10 us for 992 MB (4.2 TB/s), vector instructions issue for 60 % of a SIMD's cycles, and a wave
// waits for 69 % of its own.
#include <algorithm>
#include <cmath>

#include "mrope_rotary.h"
#include "mrope_tree.h"

namespace mrope {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kRead = 64 * 8;            // elements of a wave's read
constexpr int kReads = kWaves, kSum = kRead * kReads;  // reads, and elements, of a sum

// A probability: what is not a positive number counts as 0.
__device__ __forceinline__ double prob(float x)
{
    return __builtin_amdgcn_classf(x, 0x180) ? x : 0.0f;  // (positive and subnormal, positive and normal)
}

template <int IO>
__device__ __forceinline__ float load1(const void *p, int64_t i)
{
    if constexpr (IO == kIoF32) return static_cast<const float *>(p)[i];
    else {
        const uint16_t u = static_cast<const uint16_t *>(p)[i];
        if constexpr (IO == kIoBF16) return __uint_as_float((uint32_t)u << 16);
        else return (float)__builtin_bit_cast(_Float16, u);
    }
}

// Eight elements as they lie in memory, which begin anywhere (rows of a vocabulary are aligned to an element only).
template <int IO>
struct Eight {
    uint32_t w[IO == kIoF32 ? 8 : 4];
};

// (those before element n of them, the others 0)
template <int IO>
__device__ __forceinline__ Eight<IO> load_any(const void *p, int64_t i, int64_t n)
{
    typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
    constexpr int W = IO == kIoF32 ? 8 : 4;
    Eight<IO> x = {};
    if (n >= 8) {
        const u32x4_any *q = reinterpret_cast<const u32x4_any *>(static_cast<const char *>(p) + i * (IO == kIoF32 ? 4 : 2));
#pragma unroll
        for (int k = 0; k < W / 4; ++k) {
            const u32x4_any y = q[k];
#pragma unroll
            for (int e = 0; e < 4; ++e) x.w[4 * k + e] = y[e];
        }
    } else if (n > 0) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            if constexpr (IO == kIoF32) {
                if (e < n) x.w[e] = static_cast<const uint32_t *>(p)[i + e];
            } else {
                const uint16_t *q = static_cast<const uint16_t *>(p) + i + 2 * e;
                if (2 * e < n) x.w[e] = q[0];
                if (2 * e + 1 < n) x.w[e] |= (uint32_t)q[1] << 16;
            }
        }
    }
    return x;
}

template <int IO>
__device__ __forceinline__ void unpack_eight(const Eight<IO> &x, float (&y)[8])
{
#pragma unroll
    for (int e = 0; e < (IO == kIoF32 ? 8 : 4); ++e) {
        if constexpr (IO == kIoF32) y[e] = __uint_as_float(x.w[e]);
        else unpack16x2<IO>(x.w[e], y[2 * e], y[2 * e + 1]);
    }
}

struct Tree {  // a sequence's tokens, the first kTreeTokens of them
    int16_t parent[kTreeTokens];
    int32_t id[kTreeTokens];               // -1: not a token that can be accepted
    float p[kTreeTokens], q[kTreeTokens];  // of the parent's rows, at the token
    float u[kTreeTokens];
    Walk walk;
};
static_assert(kTreeTokens <= 32768, "parents in 16 bits");

// What the workgroup's threads tell one another.
struct Shared {
    double part[kWaves];
    int32_t hit[kWaves], last[kWaves];  // a wave's first thread that passes, its last that is not 0
    int32_t at;                         // what is found, and the sum before it
    double start;
};

struct Seq {
    int64_t t0;
    int32_t s, len, tree;  // tokens, those of the walk
};

__device__ __forceinline__ Seq seq_of(const Verify &a, int32_t s)
{
    Seq q;
    q.s = s;
    q.t0 = a.cu[s];
    q.len = (int32_t)max(min((int64_t)a.cu[s + 1], a.n_tokens) - q.t0, (int64_t)0);
    q.tree = min(q.len, kTreeTokens);
    return q;
}

template <int IO>
__device__ void load_tree(const Verify &a, const Seq &sq, Tree &t)
{
    for (int32_t i = threadIdx.x; i < sq.tree; i += kThreads) {
        const int32_t parent = a.parents ? parent_of(a.parents[sq.t0 + i], i) : i - 1;
        const int32_t id = a.ids[sq.t0 + i];
        const bool ok = parent >= 0 && id >= 0 && id < a.vocab;  // a token outside the vocabulary is not accepted
        t.parent[i] = (int16_t)parent;
        t.id[i] = ok ? id : -1;
        t.u[i] = a.u_accept[sq.t0 + i];
        t.p[i] = ok ? load1<IO>(a.target, (sq.t0 + parent) * a.target_row + id) : 0.0f;
        t.q[i] = !a.draft ? 1.0f : (ok ? load1<IO>(a.draft, (sq.t0 + parent) * a.draft_row + id) : 0.0f);
    }
}

// The first child of `node` after token `from`, or -1: a wave's search.
__device__ __forceinline__ int32_t next_child(const Tree &t, int32_t n, int32_t node, int32_t from, int lane)
{
    for (int32_t i0 = (from + 1) & ~63; i0 < n; i0 += 64) {
        const int32_t i = i0 + lane;
        const uint64_t b = __ballot(i > from && i < n && t.parent[i] == node && (t.id[i] >= 0));
        if (b) return i0 + __builtin_ctzll(b);
    }
    return -1;
}

// Whether an earlier child of the same node has token i's id (its mass is gone then).
__device__ __forceinline__ bool taken_before(const Tree &t, int32_t i, int lane)
{
    bool found = false;
    for (int32_t j0 = 0; j0 < i; j0 += 64) {
        const int32_t j = j0 + lane;
        found |= j < i && t.parent[j] == t.parent[i] && t.id[j] == t.id[i];
    }
    return __any(found);
}

// One wave: the walk on from `w` until it is over or needs the sum of its node's row (drawn drafts with a
// sibling left); `z` is that sum for the state it comes from.  The path is written by one workgroup of a sequence.
__device__ Walk go_on(const Verify &a, const Seq &sq, const Tree &t, Walk w, double z, bool writes, int lane)
{
    const bool drawn = a.draft != nullptr;
    for (;;) {
        const int32_t x = next_child(t, sq.tree, w.node, w.child, lane);
        if (x < 0) {
            w.over = 1;
            return w;
        }
        const double p = prob(t.p[x]), q = prob(t.q[x]);
        double r;
        if (drawn) r = fmax(p - w.taken * q, 0.0);
        else r = taken_before(t, x, lane) ? 0.0 : p;
        if ((double)t.u[x] * q * z < r) {
            if (writes && lane == 0) a.path[sq.t0 + w.kept] = x;
            ++w.kept;
            w.node = w.child = x;
            w.taken = 0.0;
            z = 1.0;
            continue;
        }
        w.child = x;
        if (!drawn) {
            z = fmax(z - r, 0.0);
        } else {
            w.taken += z;
            if (next_child(t, sq.tree, w.node, x, lane) >= 0) return w;
        }
    }
}

// Of the refused children of drafts that were not drawn, in a walk that is over: the ids that they have taken whole.  The
// first 64 tokens after the node are a lane each; `id_of(i)` gives what a token i has taken, -1 for one that is no child.
template <typename IdOf>
struct Gone {
    IdOf id_of;
    int32_t near;    // this lane's
    int32_t node, child;
    bool any;
    __device__ Gone(const Verify &a, const Walk &w, int lane, IdOf f) : id_of(f), near(-1), node(w.node), child(w.child)
    {
        any = !a.draft && w.child > w.node;
        if (any && w.node + 1 + lane <= w.child) near = id_of(w.node + 1 + lane);
    }
    // Takes them out of elements [at, at + kRead), eight a lane.
    __device__ __forceinline__ void out_of(int32_t at, int lane, double (&r)[8]) const
    {
        if (!any) return;
#pragma unroll 1
        for (int32_t i0 = node + 1; i0 <= child; i0 += 64) {
            int32_t id = near;
            if (i0 != node + 1) id = i0 + lane <= child ? id_of(i0 + lane) : -1;
            uint64_t b = __ballot(id >= 0 && (uint32_t)(id - at) < (uint32_t)kRead);
#pragma unroll 1
            for (; b; b &= b - 1) {
                const int d = __builtin_amdgcn_readlane(id, __builtin_ctzll(b)) - at - 8 * lane;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (d == e) r[e] = 0.0;
            }
        }
    }
};

// The values r of a lane's eight elements.
template <int IO>
__device__ __forceinline__ void row8(const Walk &w, const Eight<IO> &xp, const Eight<IO> &xq, double (&r)[8])
{
    float p[8];
    unpack_eight<IO>(xp, p);
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = prob(p[e]);
    if (w.taken > 0.0) {
        unpack_eight<IO>(xq, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = fmax(r[e] - w.taken * prob(p[e]), 0.0);
    }
}

// A lane's elements of the walk's row (0 past the vocabulary).
template <int IO>
__device__ __forceinline__ void load_row8(const Verify &a, const Seq &sq, const Walk &w, int64_t at, int lane, Eight<IO> &p, Eight<IO> &q)
{
    const int64_t tok = sq.t0 + w.node, i0 = at + 8 * lane;
    p = load_any<IO>(a.target, tok * a.target_row + i0, a.vocab - i0);
    q = Eight<IO>{};
    if (w.taken > 0.0) q = load_any<IO>(a.draft, tok * a.draft_row + i0, a.vocab - i0);
}

// Sums of the wave's lanes up to this one's.
template <int CTRL, int ROWS>
__device__ __forceinline__ double from_lane(double x)  // of the lane that CTRL names, 0 where there is none
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_scan(double x)
{
    x += from_lane<0x111, 0xF>(x);  // row_shr:1, 2, 4, 8
    x += from_lane<0x112, 0xF>(x);
    x += from_lane<0x114, 0xF>(x);
    x += from_lane<0x118, 0xF>(x);
    x += from_lane<0x142, 0xA>(x);  // row_bcast:15 and :31
    x += from_lane<0x143, 0xC>(x);
    return x;
}

// Sums over the workgroup of the threads up to this one's, and of all of them.
__device__ double block_scan(double x, double &all, Shared &sh)
{
    const double up = wave_scan(x);
    const int wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 63) sh.part[wave] = up;
    __syncthreads();
    double before = 0.0;
    all = 0.0;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
        const double y = sh.part[v];
        if (v < wave) before += y;
        all += y;
    }
    return before + up;
}

// Sums [first, end) of the walk's row, a wave each in turn, kAhead reads on their way.
template <int IO>
__device__ void row_sums(const Verify &a, const Seq &sq, const Tree &t, const Walk &w, int32_t first, int32_t end, double *sums)
{
    constexpr int kAhead = 3;  // (64 trees of 32 in bf16: 23.1 us a call, with five 24.0, eight 26.4)
    const int lane = threadIdx.x & 63;
    const Gone gone(a, w, lane, [&](int32_t i) { return t.parent[i] == w.node ? t.id[i] : -1; });
    const int32_t from = first + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int32_t n = from < end ? (end - from + kWaves - 1) / kWaves * kReads : 0;  // this wave's reads
    auto at = [&](int32_t i) { return ((int64_t)(from + i / kReads * kWaves) * kReads + i % kReads) * kRead; };
    const bool two = __builtin_amdgcn_readfirstlane(w.taken > 0.0);  // the draft's row is read too
    Eight<IO> p[kAhead] = {}, q[kAhead] = {};
    double sum = 0.0;
#pragma unroll 1
    for (int32_t i = 0; i < n + kAhead; ++i) {  // asks for read i, adds the one kAhead before
        Eight<IO> np = {}, nq = {};
        if (i < n) load_row8<IO>(a, sq, w, at(i), lane, np, nq);
        const int32_t k = i - kAhead;
        if (k >= 0) {
            double r[8];
            row8<IO>(w, p[0], q[0], r);
            gone.out_of((int32_t)min(at(k), (int64_t)a.vocab), lane, r);
            sum += ((r[0] + r[1]) + (r[2] + r[3])) + ((r[4] + r[5]) + (r[6] + r[7]));
            if (k % kReads == kReads - 1) {
                sum = wave_scan(sum);
                if (lane == 63) sums[from + k / kReads * kWaves] = sum;
                sum = 0.0;
            }
        }
#pragma unroll
        for (int j = 0; j + 1 < kAhead; ++j) p[j] = p[j + 1];
        p[kAhead - 1] = np;
        if (two) {
#pragma unroll
            for (int j = 0; j + 1 < kAhead; ++j) q[j] = q[j + 1];
            q[kAhead - 1] = nq;
        }
    }
}

struct VerifyWs {
    Walk *walk;    // [rounds][n_seqs]
    double *sums;  // [rounds][n_seqs][n_sums]
};

VerifyWs verify_ws(void *p, int32_t n_seqs, const VerifyPlan &plan)
{
    VerifyWs w;
    w.walk = static_cast<Walk *>(p);
    w.sums = reinterpret_cast<double *>(w.walk + (size_t)plan.rounds * n_seqs);
    return w;
}

// A thread's share of a row's sums: as many as the others', one after the other.
__device__ __forceinline__ double share_of(const double *sums, int32_t n)
{
    const int32_t per = (n + kThreads - 1) / kThreads, at = threadIdx.x * per;
    double x = 0.0;
#pragma unroll 1
    for (int32_t i = at; i < min(at + per, n); ++i) x += sums[i];
    return x;
}

// Sum of a row, in every thread: every workgroup of a sequence adds its parts in the same order.
__device__ double sum_of(const double *sums, int32_t n, Shared &sh)
{
    double all;
    block_scan(share_of(sums, n), all, sh);
    return all;
}

// The walk of a round, in LDS for all threads.
__device__ Walk walk_round(const Verify &a, const Seq &sq, Tree &t, Walk w, double z, bool writes)
{
    if (threadIdx.x < 64) {
        w = go_on(a, sq, t, w, z, writes, threadIdx.x);
        if (threadIdx.x == 0) t.walk = w;
    }
    __syncthreads();
    return t.walk;
}

template <int IO>
__global__ __launch_bounds__(kThreads) void verify_round_kernel(Verify a, VerifyPlan plan, VerifyWs ws, int32_t round)
{
    __shared__ Tree t;
    __shared__ Shared sh;
    const unsigned per = (unsigned)((plan.n_sums + plan.share - 1) / plan.share);  // workgroups of a sequence
    const int32_t s = (int32_t)(blockIdx.x / per), part = (int32_t)(blockIdx.x % per);
    const int64_t at = (int64_t)round * a.n_seqs + s;
    Walk w{};
    w.kept = 1;
    if (round > 0) w = ws.walk[at - a.n_seqs];  // (before it is known whether there is one)
    const Seq sq = seq_of(a, s);
    if (sq.len == 0) return;
    double z = 1.0;
    if (round > 0) {
        if (w.over) {
            if (part == 0 && threadIdx.x == 0) ws.walk[at] = w;
            return;
        }
        z = sum_of(ws.sums + (at - a.n_seqs) * plan.n_sums, plan.n_sums, sh);
    }
    load_tree<IO>(a, sq, t);
    __syncthreads();
    if (round == 0 && part == 0 && threadIdx.x == 0) a.path[sq.t0] = 0;
    w = walk_round(a, sq, t, w, z, part == 0);
    if (part == 0 && threadIdx.x == 0) {
        w.sums = round;
        ws.walk[at] = w;
    }
    row_sums<IO>(a, sq, t, w, part * plan.share, min((part + 1) * plan.share, plan.n_sums), ws.sums + at * plan.n_sums);
}

// Where the running sum of a row's sums passes u times all of them: the first that passes, else the last that holds
// anything, and the sum before it, in `sh`.  Returns the sum of all (0: nothing is found).
__device__ double find_sum(const double *sums, int32_t n, double u, Shared &sh)
{
    const int32_t per = (n + kThreads - 1) / kThreads, at = threadIdx.x * per;
    const double mine = share_of(sums, n);
    double all;
    const double run = block_scan(mine, all, sh);
    const uint64_t hit = __ballot(mine > 0.0 && run > u * all), some = __ballot(mine > 0.0);
    if ((threadIdx.x & 63) == 0) {
        const int32_t first = threadIdx.x;
        sh.hit[first >> 6] = hit ? first + __builtin_ctzll(hit) : -1;
        sh.last[first >> 6] = some ? first + 63 - __builtin_clzll(some) : -1;
    }
    __syncthreads();
    int32_t who = -1, last = -1;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
        if (who < 0) who = sh.hit[v];
        last = max(last, sh.last[v]);
    }
    if (who < 0) who = last;
    if ((int32_t)threadIdx.x == who) {  // the one of this thread's
        double before = run - mine, x;
        int32_t found = at;
#pragma unroll 1
        for (int32_t i = at; i < min(at + per, n); ++i) {
            x = sums[i];
            if (x > 0.0) found = i, sh.start = before;
            before += x;
            if (x > 0.0 && before > u * all) break;
        }
        sh.at = found;
    }
    __syncthreads();
    return all;
}

template <int IO>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(Verify a, VerifyPlan plan, VerifyWs ws)
{
    __shared__ Tree t;
    __shared__ Shared sh;
    const int32_t s = blockIdx.x;
    const int lane = threadIdx.x & 63;
    Walk w = ws.walk[(int64_t)(plan.rounds - 1) * a.n_seqs + s];  // (before it is known whether there is one)
    const double u = a.u_next[s];
    const Seq sq = seq_of(a, s);
    if (sq.len == 0) {
        if (threadIdx.x == 0) a.n_kept[s] = 0, a.next[s] = -1;
        return;
    }
    double *sums = ws.sums + ((int64_t)w.sums * a.n_seqs + s) * plan.n_sums;
    if (!w.over) {  // the rounds were not enough: the rest alone
        load_tree<IO>(a, sq, t);
        __syncthreads();
    }
    double all;
#pragma unroll 1
    for (;;) {
        if (!w.over) {  // (a walk gets further each time)
            w = walk_round(a, sq, t, w, sum_of(sums, plan.n_sums, sh), true);
        } else {
            all = find_sum(sums, plan.n_sums, u, sh);
            if (all > 0.0 || (w.taken == 0.0 && w.child == w.node)) break;
            w.taken = 0.0;  // refusals took all that the row has, to rounding: the row itself
            w.child = w.node;
        }
        row_sums<IO>(a, sq, t, w, 0, plan.n_sums, sums);
        __syncthreads();
    }
    for (int32_t i = w.kept + threadIdx.x; i < sq.len; i += kThreads) a.path[sq.t0 + i] = -1;

    // the element, a wave for each read of the sum: the first that passes, where rounding leaves none the last that is not 0
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t at = ((int64_t)sh.at * kReads + wave) * kRead;
    double r[8] = {}, sum = 0.0;
    if (all > 0.0 && at < a.vocab) {
        const Gone gone(a, w, lane, [&](int32_t i) {
            const int32_t parent = a.parents ? parent_of(a.parents[sq.t0 + i], i) : i - 1, id = a.ids[sq.t0 + i];
            return parent == w.node ? id : -1;
        });
        Eight<IO> p, q;
        load_row8<IO>(a, sq, w, at, lane, p, q);
        row8<IO>(w, p, q, r);
        gone.out_of((int32_t)at, lane, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += r[e];
    }
    double rest;
    double run = sh.start + (block_scan(sum, rest, sh) - sum);
    int first = 8, last = -1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        run += r[e];
        if (r[e] > 0.0) last = e;
        if (r[e] > 0.0 && run > u * all && first == 8) first = e;
    }
    const uint64_t hit = __ballot(first < 8), some = __ballot(last >= 0);
    const int best = 63 - __builtin_clzll(some | 1), who = hit ? __builtin_ctzll(hit) : 0;
    const int32_t h = 8 * who + __shfl(first, who), l = 8 * best + __shfl(last, best);
    if (lane == 0) {
        sh.hit[wave] = hit ? (int32_t)at + h : -1;
        sh.last[wave] = some ? (int32_t)at + l : -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int32_t next = -1;
#pragma unroll
        for (int v = kWaves - 1; v >= 0; --v) next = sh.hit[v] >= 0 ? sh.hit[v] : next;
#pragma unroll
        for (int v = kWaves - 1; v >= 0; --v) next = next < 0 ? sh.last[v] : next;
        a.n_kept[s] = w.kept;
        a.next[s] = next;
    }
}

template <int IO>
hipError_t launch_verify_io(const Verify &a, const VerifyPlan &p, const VerifyWs &ws, hipStream_t stream)
{
    for (int32_t r = 0; r < p.rounds; ++r) {
        verify_round_kernel<IO><<<dim3((unsigned)((p.n_sums + p.share - 1) / p.share) * (unsigned)a.n_seqs), kThreads, 0, stream>>>(a, p, ws, r);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    verify_pick_kernel<IO><<<dim3((unsigned)a.n_seqs), kThreads, 0, stream>>>(a, p, ws);
    return hipGetLastError();
}

}  // namespace

VerifyPlan verify_plan(int32_t n_seqs, int32_t vocab, bool drawn_trees)
{
    VerifyPlan p;
    p.rounds = drawn_trees ? 3 : 1;
    p.n_sums = (int32_t)(((int64_t)vocab + kSum - 1) / kSum);
    // about four workgroups a compute unit, each of whole turns of its waves: each repeats its sequence's walk (64 trees
    // of 32 over 248,094 ids: 24 us with two, 18 with four, 22 with eight)
    const int64_t turns = ((int64_t)p.n_sums + kWaves - 1) / kWaves;
    p.share = (int32_t)std::clamp<int64_t>((turns * n_seqs + 1023) / 1024, 1, turns) * kWaves;
    return p;
}

size_t verify_ws_bytes(int32_t n_seqs, const VerifyPlan &p)
{
    return (size_t)p.rounds * n_seqs * (sizeof(Walk) + (size_t)p.n_sums * sizeof(double));
}

hipError_t launch_verify(const Verify &a, int io, const VerifyPlan &p, void *workspace, hipStream_t stream)
{
    const VerifyWs ws = verify_ws(workspace, a.n_seqs, p);
    if (io == kIoBF16) return launch_verify_io<kIoBF16>(a, p, ws, stream);
    if (io == kIoF16) return launch_verify_io<kIoF16>(a, p, ws, stream);
    return launch_verify_io<kIoF32>(a, p, ws, stream);
}

}  // namespace mrope
