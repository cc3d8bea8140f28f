// C ABI of the 8-bit paged K/V cache: argument checks and launches of the append, the attention and
// the page calls.  The entry points are declared and documented in include/mrope.h.
#include <algorithm>
#include <cmath>
#include <numeric>
#include <utility>

#include "mrope_kv8.h"
#include "mrope_pages.h"

using namespace mrope;

namespace {

constexpr int64_t kMaxGridThreads = 0xffffffffll;  // of a launch in one dimension
constexpr int64_t kMaxContext = 1 << 27;

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

mrope_status check_kv8_shape(int32_t nk, int32_t head_dim, int32_t block_size)
{
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return fail(MROPE_ERR_UNSUPPORTED, "the 8-bit cache takes head_dim 64, 128 or 256 (got %d)", head_dim);
    if (block_size != 16 && block_size != 32 && block_size != 64)
        return fail(MROPE_ERR_UNSUPPORTED, "the 8-bit cache takes block_size 16, 32 or 64 (got %d)", block_size);
    if (nk < 1 || nk > kMaxHeads) return fail(MROPE_ERR_UNSUPPORTED, "n_kv_heads must be in [1, %d] (got %d)", kMaxHeads, nk);
    return MROPE_OK;
}

mrope_status check_kv8(const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                       int64_t num_blocks, int64_t c_block, int64_t c_tok, int64_t c_head, int32_t nk,
                       int32_t head_dim, const int32_t *tables, int64_t table_stride, int32_t table_width, int32_t n_seqs)
{
    if (num_blocks < 0 || num_blocks > 0x7fffffff) return fail(MROPE_ERR_ARG, "num_blocks out of range (%lld)", (long long)num_blocks);
    if (num_blocks > 0 && (!k_cache || !v_cache || !k_scale || !v_scale))
        return fail(MROPE_ERR_ARG, "k_cache / v_cache / k_scale / v_scale is NULL");
    if (table_width < 0 || table_stride < 0 || (n_seqs > 1 && table_stride < table_width))
        return fail(MROPE_ERR_ARG, "block_tables: table_width must be >= 0 and table_stride >= table_width");
    if (table_width > 0 && !tables) return fail(MROPE_ERR_ARG, "block_tables is NULL");
    if (c_block < 0 || c_tok < 0 || c_head < 0) return fail(MROPE_ERR_ARG, "negative stride");
    if (c_tok < head_dim || (nk > 1 && c_head < head_dim)) return fail(MROPE_ERR_ARG, "cache token / head stride < head_dim");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || c_block % 16 || c_tok % 16 || c_head % 16)
        return fail(MROPE_ERR_ALIGN, "8-bit caches must be 16-byte aligned with strides that are multiples of 16");
    if (!aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(tables, 4))
        return fail(MROPE_ERR_ALIGN, "scales and block_tables must be 4-byte aligned");
    return MROPE_OK;
}

// An append writes every row of a page from one workgroup and pages from many: rows must lie apart (by the
// strides in ascending order each past all rows of those before it).
mrope_status check_rows_apart(int64_t num_blocks, int64_t c_block, int32_t block_size, int64_t c_tok, int32_t nk, int64_t c_head,
                              int32_t head_dim)
{
    std::pair<int64_t, int64_t> dims[3] = {{c_block, num_blocks}, {c_tok, block_size}, {c_head, nk}};  // stride, extent
    std::sort(dims, dims + 3);
    int64_t span = head_dim;
    for (const auto &d : dims) {
        if (d.second <= 1) continue;
        if (d.first < span) return fail(MROPE_ERR_ARG, "cache strides: rows overlap");
        span += (d.second - 1) * d.first;
    }
    return MROPE_OK;
}

// Heads of two buffers (n_tokens x n_heads rows of head_dim elements each, element strides) that share bytes:
// views of one buffer may interleave.  Exact for one token stride; for two, tokens count as lying anywhere that
// the strides' common divisor allows.
bool heads_overlap(const void *a, int64_t a_tok, int64_t a_head, const void *b, int64_t b_tok, int64_t b_head, int32_t n_heads,
                   int64_t n_tokens, int32_t head_dim, int64_t elem_bytes)
{
    const int64_t d = (int64_t)(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) / elem_bytes;  // (16-byte aligned both)
    const int64_t a_span = (n_tokens - 1) * a_tok + (n_heads - 1) * a_head + head_dim;
    const int64_t b_span = (n_tokens - 1) * b_tok + (n_heads - 1) * b_head + head_dim;
    if (d >= a_span || -d >= b_span) return false;
    const int64_t tok = n_tokens > 1 ? std::gcd(a_tok, b_tok) : 0;
    const int64_t most = n_tokens > 1 && a_tok != b_tok ? INT64_MAX : n_tokens - 1;
    for (int32_t i = 0; i < n_heads; ++i)
        for (int32_t j = 0; j < n_heads; ++j) {
            // rows t tokens apart meet if t * tok is less than head_dim from x
            const int64_t x = d + j * b_head - i * a_head, near = tok > 0 ? x / tok : 0;
            for (int64_t t = near - 1; t <= near + 1; ++t)
                if (t >= -most && t <= most && t * tok - x < head_dim && x - t * tok < head_dim) return true;
        }
    return false;
}

Kv8 make_kv8(const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale, int64_t num_blocks,
             int64_t c_block, int64_t c_tok, int64_t c_head, int32_t nk, const int32_t *tables, int64_t table_stride,
             int32_t table_width, int32_t block_size)
{
    Kv8 kv{};
    kv.k = static_cast<uint8_t *>(const_cast<void *>(k_cache));
    kv.v = static_cast<uint8_t *>(const_cast<void *>(v_cache));
    kv.k_scale = const_cast<float *>(k_scale);
    kv.v_scale = const_cast<float *>(v_scale);
    kv.num_blocks = num_blocks;
    kv.c_block = c_block;
    kv.c_tok = c_tok;
    kv.c_head = c_head;
    kv.tables = tables;
    kv.table_stride = table_stride;
    kv.table_width = num_blocks > 0 ? table_width : 0;  // an empty pool holds nothing
    kv.block_size = block_size;
    kv.bs_shift = block_size == 16 ? 4 : (block_size == 32 ? 5 : 6);
    kv.nk = nk;
    return kv;
}

// Q, K and V of an append; n_tokens <= 2^31 - 2 keeps its grid in range too (checked by check_heads).
mrope_status check_append(void *q, int64_t q_tok, int64_t q_head, int32_t nq, const void *k, int64_t k_tok, int64_t k_head,
                          int32_t nk, const void *v, int64_t v_tok, int64_t v_head, int64_t n_tokens, int32_t head_dim,
                          int32_t rot_dim, int32_t dtype, double theta)
{
    const mrope_status st = check_heads(q, q_tok, q_head, nq, const_cast<void *>(k), k_tok, k_head, nk, n_tokens, head_dim,
                                        rot_dim, dtype, nullptr, nullptr);
    if (st != MROPE_OK) return st;
    if (!(theta > 0.0) || !std::isfinite(theta)) return fail(MROPE_ERR_ARG, "theta must be finite and > 0");
    if (n_tokens > 0 && !v) return fail(MROPE_ERR_ARG, "v is NULL");
    if (v_tok < 0 || v_head < 0) return fail(MROPE_ERR_ARG, "negative stride");
    if (nk > 1 && v_head < head_dim) return fail(MROPE_ERR_ARG, "v_head_stride < head_dim");
    const int64_t vec = dtype == MROPE_F32 ? 4 : 8;
    if (!aligned(v, 16) || v_tok % vec || v_head % vec)
        return fail(MROPE_ERR_ALIGN, "v pointer / strides break 16-byte alignment");
    return MROPE_OK;
}

Append make_append(void *q, int64_t q_tok, int64_t q_head, int32_t nq, const void *k, int64_t k_tok, int64_t k_head,
                   const void *v, int64_t v_tok, int64_t v_head, int64_t n_tokens, int32_t head_dim, int32_t n_seqs, const Kv8 &kv)
{
    Append a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_tok = q_tok;
    a.q_head = q_head;
    a.k_tok = k_tok;
    a.k_head = k_head;
    a.v_tok = v_tok;
    a.v_head = v_head;
    a.nq = nq;
    a.head_dim = head_dim;
    a.n_tokens = n_tokens;
    a.n_seqs = n_seqs;
    a.kv = kv;
    return a;
}

// The state of the page calls; fills `p`.
mrope_status check_pages(int32_t *refcount, int64_t num_blocks, int32_t *tables, int64_t table_stride, int32_t table_width,
                         int32_t *lens, int64_t n_rows, int32_t block_size, int32_t n, Pages &p)
{
    if (num_blocks < 0 || num_blocks > (1 << 24)) return fail(MROPE_ERR_ARG, "num_blocks must be in [0, 2^24] (got %lld)", (long long)num_blocks);
    if (n_rows < 0 || n_rows > (1 << 22)) return fail(MROPE_ERR_ARG, "n_rows must be in [0, 2^22] (got %lld)", (long long)n_rows);
    if (table_width < 0 || table_stride < 0 || (n_rows > 1 && table_stride < table_width))
        return fail(MROPE_ERR_ARG, "block_tables: table_width must be >= 0 and table_stride >= table_width");
    if (block_size <= 0) return fail(MROPE_ERR_ARG, "block_size must be > 0");
    if (n < 0 || n > n_rows) return fail(MROPE_ERR_ARG, "at most n_rows = %lld requests a call (got %d)", (long long)n_rows, n);
    if (num_blocks > 0 && !refcount) return fail(MROPE_ERR_ARG, "refcount is NULL");
    if (n_rows > 0 && table_width > 0 && !tables) return fail(MROPE_ERR_ARG, "block_tables is NULL");
    if (n_rows > 0 && !lens) return fail(MROPE_ERR_ARG, "seq_lens is NULL");
    if (!aligned(refcount, 4) || !aligned(tables, 4) || !aligned(lens, 4))
        return fail(MROPE_ERR_ALIGN, "refcount, block_tables and seq_lens must be 4-byte aligned");
    p = Pages{refcount, (int32_t)num_blocks, tables, table_stride, table_width, lens, (int32_t)n_rows, block_size};
    return MROPE_OK;
}

mrope_status check_pages_ws(int64_t num_blocks, int64_t n_rows, void *ws, size_t bytes)
{
    if (!ws) return fail(MROPE_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(ws, 256)) return fail(MROPE_ERR_WORKSPACE, "workspace not 256-byte aligned");
    if (bytes < pages_ws_bytes(num_blocks, n_rows))
        return fail(MROPE_ERR_WORKSPACE, "workspace too small (%zu < %zu)", bytes, pages_ws_bytes(num_blocks, n_rows));
    return MROPE_OK;
}

mrope_status check_pools(const mrope_pool *pools, int32_t n_pools, int64_t num_blocks, PoolSet &s)
{
    if (n_pools < 0 || n_pools > kMaxPools) return fail(MROPE_ERR_ARG, "n_pools must be in [0, %d] (got %d)", kMaxPools, n_pools);
    if (n_pools > 0 && !pools) return fail(MROPE_ERR_ARG, "pools is NULL");
    s = PoolSet{};
    s.n = n_pools;
    for (int32_t i = 0; i < n_pools; ++i) {
        if (!pools[i].ptr && num_blocks > 0) return fail(MROPE_ERR_ARG, "pool %d: ptr is NULL", i);
        if (pools[i].page_bytes <= 0 || pools[i].page_stride < pools[i].page_bytes)
            return fail(MROPE_ERR_ARG, "pool %d: page_bytes must be > 0 and page_stride >= page_bytes", i);
        s.ptr[i] = static_cast<char *>(pools[i].ptr);
        s.bytes[i] = pools[i].page_bytes;
        s.stride[i] = pools[i].page_stride;
        const uintptr_t all = reinterpret_cast<uintptr_t>(pools[i].ptr) | (uintptr_t)pools[i].page_bytes | (uintptr_t)pools[i].page_stride;
        s.granule[i] = all % 16 == 0 ? 16 : (all % 4 == 0 ? 4 : 1);
    }
    return MROPE_OK;
}

}  // namespace

extern "C" {

mrope_status mrope_apply_kv8(void *q, int64_t q_tok_stride, int64_t q_head_stride, int32_t n_q_heads, const void *k,
                             int64_t k_tok_stride, int64_t k_head_stride, int32_t n_kv_heads, const void *v,
                             int64_t v_tok_stride, int64_t v_head_stride, int64_t n_tokens, int32_t head_dim,
                             int32_t rot_dim, int32_t dtype, const int32_t *planes, int64_t plane_stride, double theta,
                             const int32_t *cu_seqlens, int32_t n_seqs, const int32_t *pos_offset,
                             const int32_t *block_tables, int64_t table_stride, int32_t table_width, void *k_cache,
                             void *v_cache, float *k_scale, float *v_scale, int32_t block_size, int64_t num_blocks,
                             int64_t cache_block_stride, int64_t cache_tok_stride, int64_t cache_head_stride, void *stream)
{
    mrope_status st = check_kv8_shape(n_kv_heads, head_dim, block_size);
    if (st != MROPE_OK) return st;
    st = check_append(q, q_tok_stride, q_head_stride, n_q_heads, k, k_tok_stride, k_head_stride, n_kv_heads, v, v_tok_stride,
                      v_head_stride, n_tokens, head_dim, rot_dim, dtype, theta);
    if (st != MROPE_OK) return st;
    if (n_seqs < 0) return fail(MROPE_ERR_ARG, "n_seqs < 0");
    if (n_seqs == 0 && n_tokens > 0) return fail(MROPE_ERR_ARG, "tokens given but no sequences");
    st = check_kv8(k_cache, v_cache, k_scale, v_scale, num_blocks, cache_block_stride, cache_tok_stride, cache_head_stride,
                   n_kv_heads, head_dim, block_tables, table_stride, table_width, n_seqs);
    if (st != MROPE_OK) return st;
    st = check_rows_apart(num_blocks, cache_block_stride, block_size, cache_tok_stride, n_kv_heads, cache_head_stride, head_dim);
    if (st != MROPE_OK) return st;
    if (n_tokens == 0) return MROPE_OK;
    if (!cu_seqlens) return fail(MROPE_ERR_ARG, "cu_seqlens is NULL");
    if (!planes) return fail(MROPE_ERR_ARG, "planes is NULL");
    if (plane_stride < n_tokens) return fail(MROPE_ERR_ARG, "plane_stride < n_tokens");
    if ((n_tokens / block_size + 2 * (int64_t)n_seqs) * block_size * 16 > kMaxGridThreads)
        return fail(MROPE_ERR_ARG, "too many tokens and sequences for a call (%lld, %d)", (long long)n_tokens, n_seqs);
    const Kv8 kv = make_kv8(k_cache, v_cache, k_scale, v_scale, num_blocks, cache_block_stride, cache_tok_stride,
                            cache_head_stride, n_kv_heads, block_tables, table_stride, table_width, block_size);
    Append a = make_append(q, q_tok_stride, q_head_stride, n_q_heads, k, k_tok_stride, k_head_stride, v, v_tok_stride,
                           v_head_stride, n_tokens, head_dim, n_seqs, kv);
    a.planes = planes;
    a.plane_stride = plane_stride;
    a.cu = cu_seqlens;
    a.pos = pos_offset;
    (void)hipGetLastError();
    return hip_status(launch_append(a, make_rotary(theta), dtype, static_cast<hipStream_t>(stream)), "mrope_apply_kv8");
}

mrope_status mrope_decode_kv8(void *q, int64_t q_tok_stride, int64_t q_head_stride, int32_t n_q_heads, const void *k,
                              int64_t k_tok_stride, int64_t k_head_stride, int32_t n_kv_heads, const void *v,
                              int64_t v_tok_stride, int64_t v_head_stride, int32_t n_seqs, const int32_t *pos,
                              const int32_t *amount, const int32_t *block_tables, int64_t table_stride,
                              int32_t table_width, void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                              int32_t block_size, int64_t num_blocks, int64_t cache_block_stride, int64_t cache_tok_stride,
                              int64_t cache_head_stride, int32_t head_dim, int32_t rot_dim, int32_t dtype, double theta,
                              void *stream)
{
    mrope_status st = check_kv8_shape(n_kv_heads, head_dim, block_size);
    if (st != MROPE_OK) return st;
    if (n_seqs < 0) return fail(MROPE_ERR_ARG, "n_seqs < 0");
    st = check_append(q, q_tok_stride, q_head_stride, n_q_heads, k, k_tok_stride, k_head_stride, n_kv_heads, v, v_tok_stride,
                      v_head_stride, n_seqs, head_dim, rot_dim, dtype, theta);
    if (st != MROPE_OK) return st;
    st = check_kv8(k_cache, v_cache, k_scale, v_scale, num_blocks, cache_block_stride, cache_tok_stride, cache_head_stride,
                   n_kv_heads, head_dim, block_tables, table_stride, table_width, n_seqs);
    if (st != MROPE_OK) return st;
    st = check_rows_apart(num_blocks, cache_block_stride, block_size, cache_tok_stride, n_kv_heads, cache_head_stride, head_dim);
    if (st != MROPE_OK) return st;
    if (n_seqs == 0) return MROPE_OK;
    if (!pos || !amount) return fail(MROPE_ERR_ARG, "pos / amount is NULL");
    if ((int64_t)n_seqs * block_size * 16 > kMaxGridThreads) return fail(MROPE_ERR_ARG, "too many sequences (%d)", n_seqs);
    const Kv8 kv = make_kv8(k_cache, v_cache, k_scale, v_scale, num_blocks, cache_block_stride, cache_tok_stride,
                            cache_head_stride, n_kv_heads, block_tables, table_stride, table_width, block_size);
    Append a = make_append(q, q_tok_stride, q_head_stride, n_q_heads, k, k_tok_stride, k_head_stride, v, v_tok_stride,
                           v_head_stride, n_seqs, head_dim, n_seqs, kv);
    a.pos = pos;
    a.amount = amount;
    (void)hipGetLastError();
    return hip_status(launch_append(a, make_rotary(theta), dtype, static_cast<hipStream_t>(stream)), "mrope_decode_kv8");
}

size_t mrope_attend_kv8_workspace_bytes(int64_t n_tokens, int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads,
                                        int32_t head_dim, int32_t dtype, int32_t one_token, int32_t table_width,
                                        int32_t block_size)
{
    if (n_tokens <= 0 || n_seqs <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads || table_width <= 0 ||
        block_size <= 0)
        return 0;
    return attend_workspace_bytes(n_tokens, n_seqs, n_q_heads, n_kv_heads, head_dim, dtype, one_token != 0, table_width, block_size);
}

mrope_status mrope_attend_kv8(const void *q, int64_t q_tok_stride, int64_t q_head_stride, int32_t n_q_heads,
                              int64_t n_tokens, int32_t n_kv_heads, int32_t head_dim, int32_t dtype,
                              const int32_t *cu_seqlens, int32_t n_seqs, const int32_t *context_lens,
                              const int32_t *block_tables, int64_t table_stride, int32_t table_width, const void *k_cache,
                              const void *v_cache, const float *k_scale, const float *v_scale, int32_t block_size,
                              int64_t num_blocks, int64_t cache_block_stride, int64_t cache_tok_stride,
                              int64_t cache_head_stride, double softmax_scale, void *out, int64_t out_tok_stride,
                              int64_t out_head_stride, float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    mrope_status st = check_kv8_shape(n_kv_heads, head_dim, block_size);
    if (st != MROPE_OK) return st;
    if (n_q_heads <= 0 || n_q_heads > kMaxHeads || n_q_heads % n_kv_heads)
        return fail(MROPE_ERR_UNSUPPORTED, "n_q_heads must be a multiple of n_kv_heads in [1, %d] (got %d, %d)", kMaxHeads,
                    n_q_heads, n_kv_heads);
    // Q, then the output in the place of K heads of the same count
    st = check_heads(const_cast<void *>(q), q_tok_stride, q_head_stride, n_q_heads, out, out_tok_stride, out_head_stride,
                     n_q_heads, n_tokens, head_dim, 64, dtype, nullptr, nullptr);
    if (st != MROPE_OK) return st;
    if (n_seqs < 0) return fail(MROPE_ERR_ARG, "n_seqs < 0");
    if (n_seqs == 0 && n_tokens > 0) return fail(MROPE_ERR_ARG, "tokens given but no sequences");
    if (!cu_seqlens && n_tokens != n_seqs) return fail(MROPE_ERR_ARG, "without cu_seqlens there is one token a sequence");
    const float scale_log2 = (float)(softmax_scale * 1.4426950408889634);
    if (!std::isfinite(scale_log2)) return fail(MROPE_ERR_ARG, "softmax_scale must be finite (in fp32)");
    st = check_kv8(k_cache, v_cache, k_scale, v_scale, num_blocks, cache_block_stride, cache_tok_stride, cache_head_stride,
                   n_kv_heads, head_dim, block_tables, table_stride, table_width, n_seqs);
    if (st != MROPE_OK) return st;
    if (!aligned(lse, 4)) return fail(MROPE_ERR_ALIGN, "lse must be 4-byte aligned");
    // a tile has 256 threads, and at least 4 rows, or 128 in a grid of all KV heads
    const int64_t group = n_q_heads / n_kv_heads;
    if ((n_tokens * ((group + 3) / 4) + n_seqs + 1024) * 256 > kMaxGridThreads ||
        (n_tokens * group / 128 + n_seqs) * n_kv_heads * 256 > kMaxGridThreads)
        return fail(MROPE_ERR_ARG, "too many query rows (%lld tokens, %d heads a KV head)", (long long)n_tokens, (int)group);
    if ((int64_t)table_width * block_size > kMaxContext)
        return fail(MROPE_ERR_ARG, "block_tables: at most 2^27 positions a sequence (got %lld)", (long long)table_width * block_size);
    if (n_tokens == 0) return MROPE_OK;
    if (!context_lens) return fail(MROPE_ERR_ARG, "context_lens is NULL");
    const size_t need = mrope_attend_kv8_workspace_bytes(n_tokens, n_seqs, n_q_heads, n_kv_heads, head_dim, dtype,
                                                         cu_seqlens == nullptr, num_blocks > 0 ? table_width : 0, block_size);
    if (need > 0) {
        if (!workspace) return fail(MROPE_ERR_WORKSPACE, "workspace is NULL");
        if (!aligned(workspace, 256)) return fail(MROPE_ERR_WORKSPACE, "workspace not 256-byte aligned");
        if (workspace_bytes < need) return fail(MROPE_ERR_WORKSPACE, "workspace too small (%zu < %zu)", workspace_bytes, need);
    }
    if (heads_overlap(q, q_tok_stride, q_head_stride, out, out_tok_stride, out_head_stride, n_q_heads, n_tokens, head_dim,
                      dtype == MROPE_F32 ? 4 : 2))
        return fail(MROPE_ERR_ARG, "out must not overlap q");
    Attend a{};
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.q_tok = q_tok_stride;
    a.q_head = q_head_stride;
    a.o_tok = out_tok_stride;
    a.o_head = out_head_stride;
    a.nq = n_q_heads;
    a.head_dim = head_dim;
    a.n_tokens = n_tokens;
    a.cu = cu_seqlens;
    a.n_seqs = n_seqs;
    a.ctx = context_lens;
    a.scale_log2 = scale_log2;
    a.workspace = workspace;
    a.kv = make_kv8(k_cache, v_cache, k_scale, v_scale, num_blocks, cache_block_stride, cache_tok_stride, cache_head_stride,
                    n_kv_heads, block_tables, table_stride, table_width, block_size);
    (void)hipGetLastError();
    return hip_status(launch_attend(a, dtype, static_cast<hipStream_t>(stream)), "mrope_attend_kv8");
}

size_t mrope_pages_workspace_bytes(int64_t num_blocks, int64_t n_rows)
{
    return pages_ws_bytes(num_blocks > 0 ? num_blocks : 0, n_rows > 0 ? n_rows : 0);
}

mrope_status mrope_pages_grow(int32_t *refcount, int64_t num_blocks, int32_t *block_tables, int64_t table_stride,
                              int32_t table_width, int32_t *seq_lens, int64_t n_rows, int32_t block_size,
                              const int32_t *rows, const int32_t *new_lens, int32_t n, int32_t *status, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    Pages p;
    mrope_status st = check_pages(refcount, num_blocks, block_tables, table_stride, table_width, seq_lens, n_rows, block_size, n, p);
    if (st != MROPE_OK) return st;
    if (n == 0) return MROPE_OK;
    if (!rows || !new_lens || !status) return fail(MROPE_ERR_ARG, "rows / new_lens / status is NULL");
    if ((st = check_pages_ws(num_blocks, n_rows, workspace, workspace_bytes)) != MROPE_OK) return st;
    (void)hipGetLastError();
    return hip_status(launch_pages_grow(p, rows, new_lens, n, status, pages_ws(workspace, num_blocks, n_rows),
                                        static_cast<hipStream_t>(stream)), "mrope_pages_grow");
}

mrope_status mrope_pages_free(int32_t *refcount, int64_t num_blocks, int32_t *block_tables, int64_t table_stride,
                              int32_t table_width, int32_t *seq_lens, int64_t n_rows, const int32_t *rows, int32_t n,
                              void *stream)
{
    Pages p;
    const mrope_status st = check_pages(refcount, num_blocks, block_tables, table_stride, table_width, seq_lens, n_rows, 1, n, p);
    if (st != MROPE_OK) return st;
    if (n == 0) return MROPE_OK;
    if (!rows) return fail(MROPE_ERR_ARG, "rows is NULL");
    (void)hipGetLastError();
    return hip_status(launch_pages_free(p, rows, n, static_cast<hipStream_t>(stream)), "mrope_pages_free");
}

mrope_status mrope_pages_fork(int32_t *refcount, int64_t num_blocks, int32_t *block_tables, int64_t table_stride,
                              int32_t table_width, int32_t *seq_lens, int64_t n_rows, int32_t block_size,
                              const int32_t *src, const int32_t *dst, int32_t n, int32_t *status,
                              const mrope_pool *pools, int32_t n_pools, void *workspace, size_t workspace_bytes,
                              void *stream)
{
    Pages p;
    PoolSet set;
    mrope_status st = check_pages(refcount, num_blocks, block_tables, table_stride, table_width, seq_lens, n_rows, block_size, n, p);
    if (st != MROPE_OK) return st;
    if ((st = check_pools(pools, n_pools, num_blocks, set)) != MROPE_OK) return st;
    if (n == 0) return MROPE_OK;
    if (!src || !dst || !status) return fail(MROPE_ERR_ARG, "src / dst / status is NULL");
    if ((st = check_pages_ws(num_blocks, n_rows, workspace, workspace_bytes)) != MROPE_OK) return st;
    (void)hipGetLastError();
    return hip_status(launch_pages_fork(p, src, dst, n, status, set, pages_ws(workspace, num_blocks, n_rows),
                                        static_cast<hipStream_t>(stream)), "mrope_pages_fork");
}

mrope_status mrope_pages_compact(int32_t *refcount, int64_t num_blocks, int32_t *block_tables, int64_t table_stride,
                                 int32_t table_width, int32_t *seq_lens, int64_t n_rows, int32_t *moved,
                                 const mrope_pool *pools, int32_t n_pools, void *workspace, size_t workspace_bytes,
                                 void *stream)
{
    Pages p;
    PoolSet set;
    mrope_status st = check_pages(refcount, num_blocks, block_tables, table_stride, table_width, seq_lens, n_rows, 1, 0, p);
    if (st != MROPE_OK) return st;
    if ((st = check_pools(pools, n_pools, num_blocks, set)) != MROPE_OK) return st;
    if (!moved) return fail(MROPE_ERR_ARG, "moved is NULL");
    if ((st = check_pages_ws(num_blocks, n_rows, workspace, workspace_bytes)) != MROPE_OK) return st;
    (void)hipGetLastError();
    return hip_status(launch_pages_compact(p, set, moved, pages_ws(workspace, num_blocks, n_rows),
                                           static_cast<hipStream_t>(stream)), "mrope_pages_compact");
}

mrope_status mrope_pages_copy(const mrope_pool *pools, int32_t n_pools, int64_t num_blocks, const int32_t *src,
                              const int32_t *dst, int32_t n, void *stream)
{
    PoolSet set;
    if (num_blocks < 0 || num_blocks > (1 << 24)) return fail(MROPE_ERR_ARG, "num_blocks must be in [0, 2^24] (got %lld)", (long long)num_blocks);
    const mrope_status st = check_pools(pools, n_pools, num_blocks, set);
    if (st != MROPE_OK) return st;
    if (n < 0) return fail(MROPE_ERR_ARG, "n < 0");
    if (n == 0 || n_pools == 0 || num_blocks == 0) return MROPE_OK;
    if (!src || !dst) return fail(MROPE_ERR_ARG, "src / dst is NULL");
    (void)hipGetLastError();
    return hip_status(launch_pages_copy(set, (int32_t)num_blocks, src, dst, n, static_cast<hipStream_t>(stream)), "mrope_pages_copy");
}

}  // extern "C"
