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
// chunks over workgroups.  Every workgroup of a sequence does the walk for itself (tests of single elements, fetched
// side by side for all tokens), so nothing waits for another workgroup.  The last launch finds the chunk and the
// element; walks that the rounds did not end it ends by itself, one workgroup a sequence.
// Bound: the rows' bytes, and latency where sequences are few.
#include <algorithm>
#include <cmath>

#include "mrope_rotary.h"
#include "mrope_tree.h"

namespace mrope {
namespace {

constexpr int kThreads = 256, kStep = kThreads * 8;  // elements that a workgroup reads at a time

// A probability: what is not a positive number counts as 0.
__device__ __forceinline__ double prob(float x) { return x > 0.0f && x <= 3.402823466e38f ? (double)x : 0.0; }

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

// Eight elements that begin anywhere (rows of a vocabulary are aligned to an element only).
template <int IO>
__device__ __forceinline__ void load_any8(const void *p, int64_t i, float (&x)[8])
{
    typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
    if constexpr (IO == kIoF32) {
        const u32x4_any *q = reinterpret_cast<const u32x4_any *>(static_cast<const float *>(p) + i);
        const u32x4_any a = q[0], b = q[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = __uint_as_float(a[e]);
            x[4 + e] = __uint_as_float(b[e]);
        }
    } else {
        const u32x4_any a = *reinterpret_cast<const u32x4_any *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack16x2<IO>(a[e], x[2 * e], x[2 * e + 1]);
    }
}

struct Tree {  // a sequence's tokens, the first kTreeTokens of them
    int32_t parent[kTreeTokens], id[kTreeTokens];
    float u[kTreeTokens], p[kTreeTokens], q[kTreeTokens];  // p, q: of the parent's rows, at the token
    int32_t gone[kTreeTokens], n_gone;  // ids that refused children have taken whole, of the elements in question
    double part[kThreads / 64];
    Walk walk;
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
        t.parent[i] = parent;
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

// The values r of elements i0 .. i0 + 7 of the walk's row (0 past the vocabulary), after list_gone of a range that
// holds them.
template <int IO>
__device__ __forceinline__ void row8(const Verify &a, const Seq &sq, const Tree &t, const Walk &w, int64_t i0, double (&r)[8])
{
    const int64_t tok = sq.t0 + w.node;
    const bool draft = w.taken > 0.0;
    float p[8], q[8];
    if (i0 + 8 <= a.vocab) {
        load_any8<IO>(a.target, tok * a.target_row + i0, p);
        if (draft) load_any8<IO>(a.draft, tok * a.draft_row + i0, q);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = i0 + e < a.vocab ? load1<IO>(a.target, tok * a.target_row + i0 + e) : 0.0f;
            if (draft) q[e] = i0 + e < a.vocab ? load1<IO>(a.draft, tok * a.draft_row + i0 + e) : 0.0f;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        r[e] = prob(p[e]);
        if (draft) r[e] = fmax(r[e] - w.taken * prob(q[e]), 0.0);
    }
    for (int32_t k = 0; k < t.n_gone; ++k) {
        const int64_t d = t.gone[k] - i0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (d == e) r[e] = 0.0;
    }
}

// The ids in [from, to) that the refused children have taken (drafts that were not drawn).
__device__ void list_gone(const Verify &a, Tree &t, const Walk &w, int64_t from, int64_t to)
{
    __syncthreads();
    if (threadIdx.x == 0) t.n_gone = 0;
    __syncthreads();
    if (!a.draft) {
        for (int32_t i = w.node + 1 + threadIdx.x; i <= w.child; i += kThreads)
            if (t.parent[i] == w.node && t.id[i] >= from && t.id[i] < to) t.gone[atomicAdd(&t.n_gone, 1)] = t.id[i];
    }
    __syncthreads();
}

// Sum over the workgroup, in every thread.
__device__ double block_sum(double x, Tree &t)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) t.part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) x += t.part[w];
    return x;
}

// Sum of elements [from, to) of the walk's row, in every thread.
template <int IO>
__device__ double row_sum(const Verify &a, const Seq &sq, Tree &t, const Walk &w, int64_t from, int64_t to)
{
    list_gone(a, t, w, from, to);
    double sum = 0.0;
    for (int64_t i0 = from + threadIdx.x * 8; i0 < to; i0 += kStep) {
        double r[8];
        row8<IO>(a, sq, t, w, i0, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += r[e];
    }
    return block_sum(sum, t);
}

struct VerifyWs {
    Walk *walk;    // [rounds][n_seqs]
    double *sums;  // [rounds][n_seqs][n_chunks]
};

VerifyWs verify_ws(void *p, int32_t n_seqs, const VerifyPlan &plan)
{
    VerifyWs w;
    w.walk = static_cast<Walk *>(p);
    w.sums = reinterpret_cast<double *>(w.walk + (size_t)plan.rounds * n_seqs);
    return w;
}

// Sum of a state's chunks: every workgroup of a sequence adds them in the same order.
__device__ double sum_chunks(const double *sums, int32_t n, Tree &t)
{
    double x = 0.0;
    for (int32_t i = threadIdx.x; i < n; i += kThreads) x += sums[i];
    return block_sum(x, t);
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
    const int32_t s = (int32_t)(blockIdx.x / (unsigned)plan.n_chunks), chunk = (int32_t)(blockIdx.x % (unsigned)plan.n_chunks);
    const Seq sq = seq_of(a, s);
    if (sq.len == 0) return;
    const int64_t at = (int64_t)round * a.n_seqs + s;
    double z = 1.0;
    Walk w{};
    w.kept = 1;
    if (round > 0) {
        w = ws.walk[at - a.n_seqs];
        if (w.over) {
            if (chunk == 0 && threadIdx.x == 0) ws.walk[at] = w;
            return;
        }
        z = sum_chunks(ws.sums + (at - a.n_seqs) * plan.n_chunks, plan.n_chunks, t);
    }
    load_tree<IO>(a, sq, t);
    __syncthreads();
    if (round == 0 && chunk == 0 && threadIdx.x == 0) a.path[sq.t0] = 0;
    w = walk_round(a, sq, t, w, z, chunk == 0);
    const int64_t from = (int64_t)chunk * plan.chunk, to = min(from + plan.chunk, (int64_t)a.vocab);
    const double sum = row_sum<IO>(a, sq, t, w, from, to);
    if (threadIdx.x == 0) {
        ws.sums[at * plan.n_chunks + chunk] = sum;
        w.sums = round;
        if (chunk == 0) ws.walk[at] = w;
    }
}

// Sums of the threads up to this one's and of all of them.
__device__ __forceinline__ double block_scan(double x, double &all, Tree &t)
{
    double up = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(up, o);
        if ((int)(threadIdx.x & 63) >= o) up += y;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 63) t.part[threadIdx.x >> 6] = up;
    __syncthreads();
    double before = 0.0;
    all = 0.0;
#pragma unroll
    for (int v = 0; v < kThreads / 64; ++v) {
        if (v < (int)(threadIdx.x >> 6)) before += t.part[v];
        all += t.part[v];
    }
    return before + up;
}

struct Found {
    int32_t hit, last;  // the first that passes, the last that is not 0
    double start;       // sum before it
};

constexpr int32_t kNone = 0x7fffffff;

// The first chunk whose running sum passes `want`, else the last that holds anything, and the sum before it.
__device__ int32_t find_chunk(const double *sums, int32_t n, double want, Tree &t, Found &f)
{
    if (threadIdx.x == 0) f.hit = kNone, f.last = 0, f.start = 0.0;
    double before = 0.0, all;
    for (int32_t b = 0; b < n; b += kThreads) {
        const int32_t i = b + threadIdx.x;
        const double x = i < n ? sums[i] : 0.0;
        const double run = before + block_scan(x, all, t);
        if (x > 0.0 && run > want) atomicMin(&f.hit, i);
        if (x > 0.0) atomicMax(&f.last, i);
        __syncthreads();
        if (i == (f.hit != kNone ? f.hit : f.last)) f.start = run - x;
        __syncthreads();
        if (f.hit != kNone) return f.hit;
        before += all;
    }
    return f.last;
}

// The first element of [from, to) whose running sum, begun at `before`, passes `want`; where rounding leaves none,
// the last that is not 0; -1 where all are.
template <int IO>
__device__ int32_t find_element(const Verify &a, const Seq &sq, Tree &t, const Walk &w, int64_t from, int64_t to, double before,
                                double want, Found &f)
{
    list_gone(a, t, w, from, to);
    if (threadIdx.x == 0) f.hit = kNone, f.last = -1;
    for (int64_t b = from; b < to; b += kStep) {
        const int64_t i0 = b + threadIdx.x * 8;
        double r[8] = {}, all;
        if (i0 < to) row8<IO>(a, sq, t, w, i0, r);
        double sum = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += r[e];
        double run = before + (block_scan(sum, all, t) - sum);
        int32_t first = kNone, some = -1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            run += r[e];
            if (r[e] > 0.0) {
                some = (int32_t)(i0 + e);
                if (run > want && first == kNone) first = (int32_t)(i0 + e);
            }
        }
        if (first != kNone) atomicMin(&f.hit, first);
        if (some >= 0) atomicMax(&f.last, some);
        __syncthreads();
        if (f.hit != kNone) return f.hit;
        before += all;
    }
    return f.last;
}

template <int IO>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(Verify a, VerifyPlan plan, VerifyWs ws)
{
    __shared__ Tree t;
    const int32_t s = blockIdx.x;
    const Seq sq = seq_of(a, s);
    if (sq.len == 0) {
        if (threadIdx.x == 0) a.n_kept[s] = 0, a.next[s] = -1;
        return;
    }
    const int64_t last_round = (int64_t)(plan.rounds - 1) * a.n_seqs + s;
    Walk w = ws.walk[last_round];
    load_tree<IO>(a, sq, t);
    const double *sums = ws.sums + ((int64_t)w.sums * a.n_seqs + s) * plan.n_chunks;
    double total = sum_chunks(sums, plan.n_chunks, t);
    bool chunked = true;
    while (!w.over) {  // (a walk gets further each time)
        w = walk_round(a, sq, t, w, total, true);
        total = row_sum<IO>(a, sq, t, w, 0, a.vocab);
        chunked = false;
    }
    if (!(total > 0.0)) {  // (refusals took all that the row has, to rounding)
        w.taken = 0.0;
        w.child = w.node;
        total = row_sum<IO>(a, sq, t, w, 0, a.vocab);
        chunked = false;
    }
    const double want = (double)a.u_next[s] * total;
    int64_t from = 0, to = a.vocab;
    double before = 0.0;
    __shared__ Found f;
    if (chunked) {
        from = (int64_t)find_chunk(sums, plan.n_chunks, want, t, f) * plan.chunk;
        to = min(from + plan.chunk, (int64_t)a.vocab);
        before = f.start;
    }
    const int32_t next = find_element<IO>(a, sq, t, w, from, to, before, want, f);
    if (threadIdx.x == 0) {
        a.n_kept[s] = w.kept;
        a.next[s] = next;
    }
    for (int32_t i = w.kept + threadIdx.x; i < sq.len; i += kThreads) a.path[sq.t0 + i] = -1;
}

template <int IO>
hipError_t launch_verify_io(const Verify &a, const VerifyPlan &p, const VerifyWs &ws, hipStream_t stream)
{
    for (int32_t r = 0; r < p.rounds; ++r) {
        verify_round_kernel<IO><<<dim3((unsigned)p.n_chunks * (unsigned)a.n_seqs), kThreads, 0, stream>>>(a, p, ws, r);
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
    const int64_t want = std::max<int64_t>(1, 2048 / std::max(n_seqs, 1));
    const int64_t steps = (vocab + kStep - 1) / kStep;
    p.chunk = (int32_t)std::min<int64_t>(4, std::max<int64_t>(1, steps / want)) * kStep;
    p.n_chunks = (int32_t)((vocab + p.chunk - 1) / p.chunk);
    return p;
}

size_t verify_ws_bytes(int32_t n_seqs, const VerifyPlan &p)
{
    return (size_t)p.rounds * n_seqs * (sizeof(Walk) + (size_t)p.n_chunks * sizeof(double));
}

hipError_t launch_verify(const Verify &a, int io, const VerifyPlan &p, void *workspace, hipStream_t stream)
{
    const VerifyWs ws = verify_ws(workspace, a.n_seqs, p);
    if (io == kIoBF16) return launch_verify_io<kIoBF16>(a, p, ws, stream);
    if (io == kIoF16) return launch_verify_io<kIoF16>(a, p, ws, stream);
    return launch_verify_io<kIoF32>(a, p, ws, stream);
}

}  // namespace mrope
