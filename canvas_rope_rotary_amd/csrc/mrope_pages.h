// Page management of the paged caches: launch interface (see include/mrope.h for what each call does).
#pragma once

#include "mrope_internal.h"

namespace mrope {

constexpr int kMaxPools = MROPE_MAX_POOLS;

struct PoolSet {
    char *ptr[kMaxPools];
    int64_t stride[kMaxPools];     // bytes from one page to the next
    int64_t bytes[kMaxPools];      // bytes of a page
    uint8_t granule[kMaxPools];    // bytes a lane copies at a time: 16, 4 or 1
    int32_t n;
};

struct Pages {
    int32_t *refcount;             // [num_blocks], 0 = free
    int32_t num_blocks;
    int32_t *tables;               // [n_rows][table_stride], -1 = no page
    int64_t table_stride;
    int32_t table_width;
    int32_t *lens;                 // [n_rows]
    int32_t n_rows;
    int32_t block_size;
};

// Workspace: 32-bit words, each array padded to 64 of them.
struct PagesWs {
    int32_t *head;     // [0] pages or pairs found by the plan
    int32_t *claim;    // [n_rows] first request that names the row
    int32_t *full;     // [n_rows] per request: grow: first page index wanted; fork: shared pages
    int32_t *first;    // [n_rows] per request: place of its pages in `list`, -1 = refused
    int32_t *list;     // [num_blocks] free pages (grow, fork) or holes (compact)
    int32_t *from;     // [num_blocks] compact: the page that goes to list[i]; fork: the page copied to it
    int32_t *remap;    // [num_blocks] compact: where each page goes
};

inline size_t pages_ws_words(int64_t n) { return (size_t)((n + 63) / 64 * 64); }
inline size_t pages_ws_bytes(int64_t num_blocks, int64_t n_rows)
{
    return 4 * (64 + 3 * pages_ws_words(n_rows) + 3 * pages_ws_words(num_blocks));
}
inline PagesWs pages_ws(void *p, int64_t num_blocks, int64_t n_rows)
{
    int32_t *w = static_cast<int32_t *>(p);
    const size_t r = pages_ws_words(n_rows), b = pages_ws_words(num_blocks);
    PagesWs s;
    s.head = w;
    s.claim = w + 64;
    s.full = s.claim + r;
    s.first = s.full + r;
    s.list = s.first + r;
    s.from = s.list + b;
    s.remap = s.from + b;
    return s;
}

hipError_t launch_pages_free(const Pages &p, const int32_t *rows, int32_t n, hipStream_t stream);
hipError_t launch_pages_grow(const Pages &p, const int32_t *rows, const int32_t *new_lens, int32_t n, int32_t *status,
                             const PagesWs &ws, hipStream_t stream);
hipError_t launch_pages_fork(const Pages &p, const int32_t *src, const int32_t *dst, int32_t n, int32_t *status,
                             const PoolSet &pools, const PagesWs &ws, hipStream_t stream);
hipError_t launch_pages_compact(const Pages &p, const PoolSet &pools, int32_t *moved, const PagesWs &ws, hipStream_t stream);
hipError_t launch_pages_copy(const PoolSet &pools, int32_t num_blocks, const int32_t *src, const int32_t *dst, int32_t n,
                             hipStream_t stream);

}  // namespace mrope
