// The paged K/V cache in 8 bits: what the append and the attention kernels share.
//
// Element (block, row, head, d) of either cache is one e4m3 byte at block*c_block + row*c_tok +
// head*c_head + d, and stands for code * scale[block*nk + head].  Scales are powers of two: dividing
// by one is exact, so a value is rounded once, to e4m3, and a page whose scale grows is re-coded by
// an exact shift of the exponent (codes lose bits only where they fall below e4m3's normal range).
#pragma once

#include "mrope_internal.h"

namespace mrope {

constexpr int kMinScaleExp = -96, kMaxScaleExp = 120;

struct Kv8 {
    uint8_t *k, *v;
    float *k_scale, *v_scale;  // [num_blocks][nk]
    int64_t num_blocks;
    int64_t c_block, c_tok, c_head;  // in bytes (one byte an element)
    const int32_t *tables;     // [n_seqs][table_stride]: the pages of each sequence, in order
    int64_t table_stride;
    int32_t table_width;       // entries of a row that may be read
    int32_t block_size;        // 16, 32 or 64
    int32_t bs_shift;
    int32_t nk;
};

struct Append {
    void *q;
    const void *k, *v;
    int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;
    int32_t nq, head_dim;
    int64_t n_tokens;
    const int32_t *planes;      // [3][plane_stride]; nullptr: one token a sequence at pos - amount
    int64_t plane_stride;
    const int32_t *cu;          // [n_seqs + 1]
    int32_t n_seqs;
    const int32_t *pos;         // prefill: position of each sequence's first token (nullable); decode: of its token
    const int32_t *amount;      // decode only
    Kv8 kv;
};

struct Attend {
    const void *q;
    void *out;
    float *lse;                 // nullable: [n_tokens][nq]
    int64_t q_tok, q_head, o_tok, o_head;
    int32_t nq, head_dim;
    int64_t n_tokens;
    const int32_t *cu;          // nullable: one token a sequence
    int32_t n_seqs;
    const int32_t *ctx;         // tokens of each sequence in the cache, the query tokens included
    float scale_log2;           // softmax scale * log2(e)
    void *workspace;
    Kv8 kv;
};

struct AttendTree : Attend {
    const uint64_t *mask;       // [n_tokens][mask_words]: bit j of a token's row: it sees token j of its sequence
    int32_t mask_words;
};

hipError_t launch_append(const Append &a, const Rotary &r, int io, hipStream_t stream);
size_t attend_workspace_bytes(int64_t n_tokens, int32_t n_seqs, int32_t nq, int32_t nk, int32_t head_dim, int io,
                              bool one_token, int32_t table_width, int32_t block_size);
hipError_t launch_attend(const Attend &a, int io, hipStream_t stream);
size_t attend_tree_workspace_bytes(int64_t n_tokens, int32_t n_seqs, int32_t nq, int32_t nk, int32_t head_dim, int io,
                                   int32_t table_width, int32_t block_size);
hipError_t launch_attend_tree(const AttendTree &a, int io, hipStream_t stream);

#if defined(__HIPCC__)
namespace {

// Exponent e of the smallest power of two with amax <= 448 * 2^e (448 = 1.75 * 2^8 is the largest
// e4m3 value), clamped to the range of a scale.  amax is finite and >= 0.
__device__ __forceinline__ int scale_exp_for(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, kMinScaleExp), kMaxScaleExp);
}

// The exponent of a stored scale (a power of two written by an append), clamped to its range.
__device__ __forceinline__ int scale_exp_of(float s)
{
    const int e = (int)((__float_as_uint(s) >> 23) & 0xffu) - 127;
    return min(max(e, kMinScaleExp), kMaxScaleExp);
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Four fp32 values to four e4m3 bytes, each rounded to nearest even (|x| <= 448 or NaN here).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

typedef float kv8_f32x2 __attribute__((ext_vector_type(2)));

// Four e4m3 bytes times f, rounded to e4m3 again (f: a power of two that takes none of them past 448).
__device__ __forceinline__ uint32_t shift_e4m3(uint32_t u, float f)
{
    const kv8_f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, false);
    const kv8_f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, true);
    return pack_e4m3(lo[0] * f, lo[1] * f, hi[0] * f, hi[1] * f);
}

}  // namespace
#endif

}  // namespace mrope
