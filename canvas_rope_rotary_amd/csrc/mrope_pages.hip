// Page management of the paged caches: mrope_pages_free, _grow, _fork, _compact, _copy.
//
// The state is three arrays (reference counts, block tables, lengths) and no free list: a page is
// free when its count is 0, and pages are handed out lowest index first, so every call's result is a
// function of the state alone.  A plan kernel of one workgroup ranks the free (or live) pages by a
// running prefix sum and settles which requests are granted; a wide kernel then copies table rows and
// pages.  Nothing returns to the host between them.
//
// Bound: the plans by latency (three or four rounds of memory and a prefix sum: 64 requests on 2,048 pages 6 to
// 7 us, the compaction of 16,384 pages 12 us), the copies by HBM (134 MB in 24.7 us, 5.4 TB/s).
#include <algorithm>

#include "mrope_pages.h"

namespace mrope {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kPlan = 1024;  // threads of the plan kernels
constexpr int32_t kNotEnough = 1, kBadRow = 2;  // MROPE_PAGES_*

// Exclusive prefix sum of v over the workgroup; total in `sum`.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T &sum)
{
    __shared__ T part[kPlan / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    T x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const T y = __shfl_up(x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // `part` of an earlier scan has been read
    if (lane == 63) part[wave] = x;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlan / 64; ++w) {
        const T p = part[w];
        if (w < wave) before += p;
        all += p;
    }
    sum = all;
    return before + x - v;
}

// list[rank] = page for the pages of [from, to) with (refcount > 0) == live and rank < most; returns
// how many there are below `most` or more (every page is counted until `most` are found).  A thread takes
// kPer pages at a time: 16 where all of the pool is ranked, 4 where a few pages are wanted (pages are
// few as well then, or the first thousands hold them).
template <int kPer>
__device__ int32_t rank_pages(const int32_t *ref, int32_t from, int32_t to, bool live, int32_t most, int32_t *list)
{
    int32_t found = 0;
    const bool wide = reinterpret_cast<uintptr_t>(ref) % 16 == 0;
    for (int64_t b = from / kPer * kPer; b < to && found < most; b += kPlan * kPer) {
        const int64_t p0 = b + (int64_t)threadIdx.x * kPer;
        int32_t r[kPer], c = 0;
        if (wide && p0 + kPer <= to) {
#pragma unroll
            for (int i = 0; i < kPer; i += 4) {
                const u32x4 x = *reinterpret_cast<const u32x4 *>(ref + p0 + i);
#pragma unroll
                for (int e = 0; e < 4; ++e) r[i + e] = (int32_t)x[e];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) r[i] = p0 + i < to ? ref[p0 + i] : 0;
        }
        uint32_t hit = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) hit |= ((r[i] > 0) == live && p0 + i >= from && p0 + i < to ? 1u : 0u) << i;
        c = __builtin_popcount(hit);
        int32_t sum;
        int32_t at = found + block_scan(c, sum);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (hit >> i & 1) {
                if (at < most) list[at] = (int32_t)(p0 + i);
                ++at;
            }
        found += sum;
    }
    return found;
}

__device__ __forceinline__ int32_t pages_of(int32_t len, int32_t bs) { return len > 0 ? (int32_t)(((int64_t)len + bs - 1) / bs) : 0; }

// The first request that names each row keeps it.
__device__ void claim_rows(const int32_t *rows, int32_t n, int32_t n_rows, int32_t *claim)
{
    for (int32_t i = threadIdx.x; i < n; i += kPlan)
        if (rows[i] >= 0 && rows[i] < n_rows) claim[rows[i]] = 0x7fffffff;
    __syncthreads();
    for (int32_t i = threadIdx.x; i < n; i += kPlan)
        if (rows[i] >= 0 && rows[i] < n_rows) atomicMin(&claim[rows[i]], i);
    __syncthreads();
}

// Requests in order, each wanting need(i) pages (< 0: a bad row): ws.first[i] = place of its first
// page in ws.list or -1, status[i], and ws.list filled.  A request is granted if the pages wanted up
// to and with it are free, so after one that is not, only those that want nothing are.
template <typename Need>
__device__ void plan_requests(const Pages &p, int32_t n, const PagesWs &ws, int32_t *status, Need need)
{
    int64_t wanted = 0, sum;  // (a table's width of pages for each request may pass 32 bits together)
    for (int32_t b = 0; b < n; b += kPlan) {
        const int32_t i = b + threadIdx.x;
        const int32_t want = i < n ? need(i) : 0;
        const int64_t at = block_scan((int64_t)max(want, 0), sum);
        if (i < n) ws.first[i] = want < 0 ? -1 : (int32_t)min(wanted + at, (int64_t)0x7fffffff);
        wanted += sum;
    }
    const int32_t most = (int32_t)min(wanted, (int64_t)p.num_blocks);
    const int32_t found = min(rank_pages<4>(p.refcount, 0, p.num_blocks, false, most, ws.list), most);
    __syncthreads();
    for (int32_t i = threadIdx.x; i < n; i += kPlan) {
        int32_t st = 0;
        if (ws.first[i] < 0) {
            st = kBadRow;
        } else {
            const int32_t want = need(i);
            if (want > 0 && (int64_t)ws.first[i] + want > found) {
                st = kNotEnough;
                ws.first[i] = -1;
            }
        }
        status[i] = st;
    }
    __syncthreads();
}

__global__ __launch_bounds__(256) void pages_free_kernel(Pages p, const int32_t *rows)
{
    const int32_t r = rows[blockIdx.x];
    if (r < 0 || r >= p.n_rows) return;
    int32_t *t = p.tables + r * p.table_stride;
    // the exchange gives each entry's page back once, however often the row is named
    for (int32_t i = threadIdx.x; i < p.table_width; i += 256) {
        if (t[i] == -1) continue;
        const int32_t page = atomicExch(&t[i], -1);
        if (page >= 0 && page < p.num_blocks) atomicSub(&p.refcount[page], 1);
    }
    if (threadIdx.x == 0) p.lens[r] = 0;
}

__global__ __launch_bounds__(kPlan) void pages_grow_kernel(Pages p, const int32_t *rows, const int32_t *new_lens, int32_t n,
                                                           int32_t *status, PagesWs ws)
{
    claim_rows(rows, n, p.n_rows, ws.claim);
    auto need = [&](int32_t i) {
        const int32_t r = rows[i], len = new_lens[i];
        if (r < 0 || r >= p.n_rows || ws.claim[r] != i || len < 0 || pages_of(len, p.block_size) > p.table_width) return -1;
        return max(pages_of(len, p.block_size) - pages_of(p.lens[r], p.block_size), 0);
    };
    plan_requests(p, n, ws, status, need);
    // a wave a request: its pages in order
    const int lane = threadIdx.x & 63;
    for (int32_t i = threadIdx.x >> 6; i < n; i += kPlan / 64) {
        const int32_t first = ws.first[i];
        if (first < 0) continue;
        const int32_t r = rows[i], len = p.lens[r];
        const int32_t has = pages_of(len, p.block_size), want = pages_of(new_lens[i], p.block_size);
        for (int32_t k = has + lane; k < want; k += 64) {
            const int32_t page = ws.list[first + k - has];
            p.tables[r * p.table_stride + k] = page;
            p.refcount[page] = 1;
        }
        if (lane == 0 && new_lens[i] > len) p.lens[r] = new_lens[i];
    }
}

__global__ __launch_bounds__(kPlan) void pages_fork_plan_kernel(Pages p, const int32_t *src, const int32_t *dst, int32_t n,
                                                                int32_t *status, PagesWs ws)
{
    claim_rows(dst, n, p.n_rows, ws.claim);
    auto need = [&](int32_t i) {
        const int32_t s = src[i], d = dst[i];
        if (s < 0 || s >= p.n_rows || d < 0 || d >= p.n_rows || ws.claim[d] != i || p.lens[d] != 0) return -1;
        return p.lens[s] > 0 && p.lens[s] % p.block_size && p.lens[s] / p.block_size < p.table_width ? 1 : 0;
    };
    plan_requests(p, n, ws, status, need);
    // lengths are read before any is written: a source may be another request's (empty) destination
    for (int32_t b = 0; b < n; b += kPlan) {
        const int32_t i = b + threadIdx.x;
        int32_t len = 0;
        if (i < n && ws.first[i] >= 0) len = max(p.lens[src[i]], 0);
        if (i < n) ws.full[i] = len;
    }
    __syncthreads();
    for (int32_t i = threadIdx.x; i < n; i += kPlan) {
        const int32_t first = ws.first[i];
        if (first < 0) continue;
        const int32_t len = ws.full[i], full = min(len / p.block_size, p.table_width);
        p.lens[dst[i]] = len;
        int32_t mine = -1;
        if (len % p.block_size && full < p.table_width) {  // the last page is copied, the others are shared
            mine = ws.list[first];
            p.refcount[mine] = 1;
            ws.from[first] = p.tables[src[i] * p.table_stride + full];
        }
        ws.full[i] = full;
        ws.claim[dst[i]] = mine;
    }
    // one entry of `list` and `from` a copied page: those granted are a prefix
    __shared__ int32_t copies;
    if (threadIdx.x == 0) copies = 0;
    __syncthreads();
    for (int32_t i = threadIdx.x; i < n; i += kPlan)
        if (ws.first[i] >= 0 && ws.claim[dst[i]] >= 0) atomicMax(&copies, ws.first[i] + 1);
    __syncthreads();
    if (threadIdx.x == 0) ws.head[0] = copies;
}

__global__ __launch_bounds__(kPlan) void pages_compact_plan_kernel(Pages p, int32_t *moved, PagesWs ws)
{
    int32_t c = 0, live;
#pragma unroll 8
    for (int64_t b = (int64_t)threadIdx.x; b < p.num_blocks; b += kPlan) {
        c += p.refcount[b] > 0;
        ws.remap[b] = (int32_t)b;
    }
    block_scan(c, live);
    // the i-th free page below `live` takes the i-th live page from there on: there are as many
    const int32_t n = rank_pages<16>(p.refcount, 0, live, false, p.num_blocks, ws.list);
    rank_pages<16>(p.refcount, live, p.num_blocks, true, p.num_blocks, ws.from);
    __syncthreads();
    for (int32_t i = threadIdx.x; i < n; i += kPlan) {
        const int32_t to = ws.list[i], from = ws.from[i];
        ws.remap[from] = to;
        p.refcount[to] = p.refcount[from];
        p.refcount[from] = 0;
    }
    if (threadIdx.x == 0) ws.head[0] = *moved = n;
}

// Bytes [at, end) of a page by a wave, four loads on their way at a time.
template <typename T>
__device__ __forceinline__ void copy_span(char *to, const char *from, int64_t at, int64_t end)
{
    constexpr int U = 4, kStep = 64 * sizeof(T);
    for (at += (threadIdx.x & 63) * sizeof(T); at < end; at += U * kStep) {
        T x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (at + u * kStep < end) x[u] = *reinterpret_cast<const T *>(from + at + u * kStep);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (at + u * kStep < end) *reinterpret_cast<T *>(to + at + u * kStep) = x[u];
    }
}

// Pages from[i] -> to[i] of every pool, pool after pool, a wave for kSpan bytes of a page: pages of a few
// bytes (scales) do not hold a workgroup up, and large ones are shared out.
constexpr int64_t kSpan = 4096;

__device__ void copy_pages(const PoolSet &pools, int32_t num_blocks, const int32_t *from, const int32_t *to, int32_t n,
                           int64_t block, int64_t n_blocks)
{
    const int64_t waves = n_blocks * 4;
    int64_t u = __builtin_amdgcn_readfirstlane((int)block * 4 + (threadIdx.x >> 6));
    for (int k = 0; k < pools.n; ++k) {
        const int64_t spans = (pools.bytes[k] + kSpan - 1) / kSpan, units = n * spans;
        for (; u < units; u += waves) {
            const int32_t i = (int32_t)(spans == 1 ? u : u / spans);
            const int64_t at = (u - i * spans) * kSpan, end = min(at + kSpan, pools.bytes[k]);
            const int32_t a = from[i], b = to[i];
            if (a < 0 || a >= num_blocks || b < 0 || b >= num_blocks || a == b) continue;
            char *dst = pools.ptr[k] + b * pools.stride[k];
            const char *src = pools.ptr[k] + a * pools.stride[k];
            if (pools.granule[k] == 16) copy_span<u32x4>(dst, src, at, end);
            else if (pools.granule[k] == 4) copy_span<uint32_t>(dst, src, at, end);
            else copy_span<uint8_t>(dst, src, at, end);
        }
        u -= units;  // the next pool's pages go on with the next wave
    }
}

__global__ __launch_bounds__(256) void pages_fork_kernel(Pages p, const int32_t *src, const int32_t *dst, int32_t n,
                                                         PoolSet pools, PagesWs ws)
{
    if ((int32_t)blockIdx.x < n) {  // a workgroup a request: the child's table row
        const int32_t i = blockIdx.x;
        if (ws.first[i] < 0) return;
        const int32_t *s = p.tables + src[i] * p.table_stride;
        int32_t *d = p.tables + dst[i] * p.table_stride;
        const int32_t full = ws.full[i], mine = ws.claim[dst[i]];
        for (int32_t k = threadIdx.x; k < p.table_width; k += 256) {
            int32_t page = -1;
            if (k < full) {
                page = s[k];
                if (page >= 0 && page < p.num_blocks) atomicAdd(&p.refcount[page], 1);
            } else if (k == full) {
                page = mine;
            }
            d[k] = page;
        }
        return;
    }
    copy_pages(pools, p.num_blocks, ws.from, ws.list, ws.head[0], (int64_t)blockIdx.x - n, (int64_t)gridDim.x - n);
}

__global__ __launch_bounds__(256) void pages_compact_kernel(Pages p, PoolSet pools, PagesWs ws)
{
    const int32_t n = ws.head[0];
    if (n == 0) return;
    for (int64_t r = blockIdx.x; r < p.n_rows; r += gridDim.x) {
        int32_t *t = p.tables + r * p.table_stride;
        for (int32_t k = threadIdx.x; k < p.table_width; k += 256) {
            const int32_t page = t[k];
            if (page >= 0 && page < p.num_blocks) {
                const int32_t to = ws.remap[page];
                if (to != page) t[k] = to;
            }
        }
    }
    copy_pages(pools, p.num_blocks, ws.from, ws.list, n, blockIdx.x, gridDim.x);
}

__global__ __launch_bounds__(256) void pages_copy_kernel(PoolSet pools, int32_t num_blocks, const int32_t *src,
                                                         const int32_t *dst, int32_t n)
{
    copy_pages(pools, num_blocks, src, dst, n, blockIdx.x, gridDim.x);
}

constexpr int64_t kCopyBlocks = 2048;

}  // namespace

hipError_t launch_pages_free(const Pages &p, const int32_t *rows, int32_t n, hipStream_t stream)
{
    pages_free_kernel<<<n, 256, 0, stream>>>(p, rows);
    return hipGetLastError();
}

hipError_t launch_pages_grow(const Pages &p, const int32_t *rows, const int32_t *new_lens, int32_t n, int32_t *status,
                             const PagesWs &ws, hipStream_t stream)
{
    pages_grow_kernel<<<1, kPlan, 0, stream>>>(p, rows, new_lens, n, status, ws);
    return hipGetLastError();
}

hipError_t launch_pages_fork(const Pages &p, const int32_t *src, const int32_t *dst, int32_t n, int32_t *status,
                             const PoolSet &pools, const PagesWs &ws, hipStream_t stream)
{
    pages_fork_plan_kernel<<<1, kPlan, 0, stream>>>(p, src, dst, n, status, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t copies = std::min<int64_t>((int64_t)n * pools.n, kCopyBlocks);
    pages_fork_kernel<<<(unsigned)(n + std::max<int64_t>(copies, 1)), 256, 0, stream>>>(p, src, dst, n, pools, ws);
    return hipGetLastError();
}

hipError_t launch_pages_compact(const Pages &p, const PoolSet &pools, int32_t *moved, const PagesWs &ws, hipStream_t stream)
{
    pages_compact_plan_kernel<<<1, kPlan, 0, stream>>>(p, moved, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t units = std::max<int64_t>((int64_t)p.num_blocks / 2 * pools.n, p.n_rows);
    pages_compact_kernel<<<(unsigned)std::min<int64_t>(std::max<int64_t>(units, 1), kCopyBlocks), 256, 0, stream>>>(p, pools, ws);
    return hipGetLastError();
}

hipError_t launch_pages_copy(const PoolSet &pools, int32_t num_blocks, const int32_t *src, const int32_t *dst, int32_t n,
                             hipStream_t stream)
{
    pages_copy_kernel<<<(unsigned)std::min<int64_t>((int64_t)n * pools.n, kCopyBlocks), 256, 0, stream>>>(pools, num_blocks, src, dst, n);
    return hipGetLastError();
}

}  // namespace mrope
