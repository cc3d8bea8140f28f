// Trees of drafted tokens: position planes and masks (mrope_planes_tree), and the cache's rows of an accepted path
// moved together (mrope_keep_kv8).
#include <algorithm>

#include "mrope_tree.h"

namespace mrope {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ planes and masks -----------
// A workgroup a sequence, a thread a token, the sequence's parents in LDS.  A token's ancestors come in descending
// order (a parent comes before its children), so the words of its mask are finished one after the other.
// Bound: latency, a read of LDS for each step to the root.  A tree of 8 tokens takes 2.0 us, 512 random ones of 64 4.2 and 32 of
// 1,024 17.  Deep trees take a time that grows with their depth: 512 chains of 64 10.8 us, one chain of 1,024, or 32 of
// them, 365 to 371 (a thread takes four of the tokens, 2,560 steps of some 290 cycles for the last).
constexpr int kPlanesThreads = 256;

__global__ __launch_bounds__(kPlanesThreads) void planes_tree_kernel(PlanesTree a)
{
    __shared__ int32_t parent[kTreeTokens];
    const int32_t s = blockIdx.x, t0 = a.cu[s];
    const int32_t len = (int32_t)min((int64_t)a.cu[s + 1], a.n_tokens) - t0;
    for (int32_t i = threadIdx.x; i < min(len, kTreeTokens); i += kPlanesThreads) parent[i] = parent_of(a.parents[t0 + i], i);
    const int32_t root = a.pos[s] - (a.amount ? a.amount[s] : 0);
    __syncthreads();
    for (int32_t i = threadIdx.x; i < len; i += kPlanesThreads) {
        uint64_t *row = a.mask + (int64_t)(t0 + i) * a.mask_words;
        int32_t depth = 0, w = a.mask_words - 1;
        uint64_t bits = 0;
        for (int32_t p = i; p >= 0;) {
            const int32_t at = p >> 6;
            if (at < a.mask_words) {
                for (; w > at; --w, bits = 0) row[w] = bits;
                bits |= 1ull << (p & 63);
            }
            p = p < kTreeTokens ? parent[p] : -1;
            depth += p >= 0;
        }
        for (; w >= 0; --w, bits = 0) row[w] = bits;
        const int32_t plane = root + depth;
#pragma unroll
        for (int k = 0; k < 3; ++k) a.planes[k * a.plane_stride + t0 + i] = plane;
    }
}

// ------------------------------------------------------------------ keep -----------------------
// A wave for each (sequence, layer, K or V, head): these have their own rows and scales, so nothing but the order
// of one wave's loads and stores matters.  It takes the pages that the kept rows go to in ascending order and holds
// a page's new rows in registers before it writes it: a row comes from its own position or from one further on,
// so no later page's source is overwritten.
// Bound: latency (count -> path -> table -> codes and scales -> reduction -> stores).  Six layers of 2 KV heads of 256: 8 trees of
// 16 tokens 5.2 us, 256 of 32 9.3 us, of which 8 MB of rows are 2.
template <int D, int BS>
__global__ __launch_bounds__(256) void keep_kernel(Keep a, KeepLayers layers)
{
    constexpr int LPR = D / 16;          // lanes a row, 16 codes each
    constexpr int RPL = 64 / LPR;        // rows of a load
    constexpr int NL = BS / RPL;         // loads of a page
    const Kv8 &kv = a.kv;
    const int lane = threadIdx.x & 63;
    const int32_t per = a.n_layers * 2 * kv.nk;  // units of a sequence
    const int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int32_t s = (int32_t)(u / per);
    if (s >= a.n_seqs) return;
    const int32_t unit = (int32_t)(u - (int64_t)s * per), h = unit % kv.nk;
    const bool is_v = (unit / kv.nk) & 1;
    const mrope_kv8_layer &layer = layers.at[unit / (2 * kv.nk)];
    uint8_t *cache = static_cast<uint8_t *>(is_v ? layer.v_cache : layer.k_cache) + h * kv.c_head;
    float *scales = (is_v ? layer.v_scale : layer.k_scale) + h;

    const int64_t pos = a.pos[s];
    if (pos < 0) return;
    const int32_t t0 = a.cu[s];
    const int32_t len = (int32_t)(min((int64_t)a.cu[s + 1], a.n_tokens) - t0);
    const int32_t *path = a.path + t0;
    // entries that ascend within the sequence
    int32_t m = min(a.n_kept[s], len);
    for (int32_t i0 = 0; i0 < m; i0 += 64) {
        const int32_t i = i0 + lane;
        bool bad = false;
        if (i < m) {
            const int32_t x = path[i], before = i > 0 ? path[i - 1] : -1;
            bad = x <= before || x < 0 || x >= len;
        }
        const uint64_t b = __ballot(bad);
        if (b) m = i0 + __builtin_ctzll(b);
    }

    auto page_of = [&](int64_t p) {
        const int64_t k = p >> kv.bs_shift;
        const int32_t page = k < kv.table_width ? kv.tables[s * kv.table_stride + k] : -1;
        return page >= 0 && page < kv.num_blocks ? page : -1;
    };
    const int sub = lane / LPR, piece = lane % LPR * 16;
    for (int64_t at = pos; at < pos + m;) {
        const int64_t first = at >> kv.bs_shift << kv.bs_shift;
        const int64_t end = min(pos + m, first + BS);
        const int32_t page = page_of(at);
        const int held = (int)(at - first);
        const int32_t i0 = (int32_t)(at - pos);
        at = end;
        if (page < 0) continue;
        uint8_t *to = cache + page * kv.c_block + piece;
        float *scale = scales + (int64_t)page * kv.nk;
        const int was = scale_exp_of(*scale);

        // the new rows: code and exponent
        u32x4 x[NL];
        int es[NL];
        bool mine[NL], moved[NL];
        int need = kMinScaleExp;
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            const int row = k * RPL + sub;
            mine[k] = row >= held && first + row < end;
            moved[k] = false;
            x[k] = u32x4{0, 0, 0, 0};
            es[k] = 0;
            if (!mine[k]) continue;
            const int64_t from = pos + path[i0 + row - held];
            const int32_t src = page_of(from);
            mine[k] = src >= 0;
            if (!mine[k]) continue;
            moved[k] = from != first + row;
            x[k] = *reinterpret_cast<const u32x4 *>(cache + src * kv.c_block + (from & (BS - 1)) * kv.c_tok + piece);
            es[k] = scale_exp_of(scales[(int64_t)src * kv.nk]);
        }
        bool any = false;
#pragma unroll
        for (int k = 0; k < NL; ++k) any |= mine[k];
        if (!__any(any)) continue;  // none of the rows has a page to come from
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            if (!mine[k]) continue;
            uint32_t top = 0;  // the largest code that is a number: they are in the order of their bits
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t c = x[k][w] >> (8 * b) & 0x7f;
                    if (c != 0x7f) top = max(top, c);
                }
            if (top) {
                const float v = __builtin_amdgcn_cvt_f32_fp8((int)top, 0);  // in [2^-9, 448]
                const uint32_t bits = __float_as_uint(v);
                need = max(need, es[k] + (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0));
            }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) need = max(need, __shfl_xor(need, o));
        int e = min(need, kMaxScaleExp);
        if (held > 0) {
            if (e > was) {  // the rows already here go to the larger scale
                const float f = pow2(max(was - e, -126));
                for (int row = sub; row < held; row += RPL) {
                    u32x4 *p = reinterpret_cast<u32x4 *>(to + row * kv.c_tok);
                    u32x4 y = *p;
#pragma unroll
                    for (int w = 0; w < 4; ++w) y[w] = shift_e4m3(y[w], f);
                    *p = y;
                }
            } else {
                e = was;
            }
        }
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            if (!mine[k] || (!moved[k] && es[k] == e)) continue;
            // (a number other than 0 is 2^-9 of its scale at least, so its page's is no less than 2^-17 of it; a row of zeros
            // may come from any)
            const float f = pow2(min(max(es[k] - e, -126), 17));
#pragma unroll
            for (int w = 0; w < 4; ++w) x[k][w] = shift_e4m3(x[k][w], f);
            *reinterpret_cast<u32x4 *>(to + (k * RPL + sub) * kv.c_tok) = x[k];
        }
        if (lane == 0) *scale = pow2(e);
    }
}

template <int D>
hipError_t launch_keep_d(const Keep &a, const KeepLayers &layers, unsigned grid, hipStream_t stream)
{
    switch (a.kv.block_size) {
    case 16: keep_kernel<D, 16><<<grid, 256, 0, stream>>>(a, layers); break;
    case 32: keep_kernel<D, 32><<<grid, 256, 0, stream>>>(a, layers); break;
    default: keep_kernel<D, 64><<<grid, 256, 0, stream>>>(a, layers); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_planes_tree(const PlanesTree &a, hipStream_t stream)
{
    planes_tree_kernel<<<(unsigned)a.n_seqs, kPlanesThreads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_keep(const Keep &a, const KeepLayers &layers, hipStream_t stream)
{
    const int64_t units = (int64_t)a.n_seqs * a.n_layers * 2 * a.kv.nk;
    const unsigned grid = (unsigned)((units + 3) / 4);
    switch (a.head_dim) {
    case 64: return launch_keep_d<64>(a, layers, grid, stream);
    case 128: return launch_keep_d<128>(a, layers, grid, stream);
    default: return launch_keep_d<256>(a, layers, grid, stream);
    }
}

}  // namespace mrope
