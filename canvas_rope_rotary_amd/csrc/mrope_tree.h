// Trees of drafted tokens: planes and masks, verification, and the rows of the accepted path (see include/mrope.h
// for what each call does).
#pragma once

#include "mrope_kv8.h"

namespace mrope {

constexpr int kTreeTokens = MROPE_TREE_MAX_TOKENS;

// The parent of token i, which has to come before it; -1: none.
__host__ __device__ inline int32_t parent_of(int32_t parent, int32_t i) { return parent >= 0 && parent < i ? parent : -1; }

struct PlanesTree {
    const int32_t *parents;     // [n_tokens] index in the sequence
    const int32_t *cu;          // [n_seqs + 1]
    int32_t n_seqs;
    int64_t n_tokens;
    const int32_t *pos, *amount;  // [n_seqs], amount nullable
    int32_t *planes;            // [3][plane_stride]
    int64_t plane_stride;
    uint64_t *mask;             // [n_tokens][mask_words]
    int32_t mask_words;
};

struct Verify {
    const void *target, *draft;  // [n_tokens][vocab], rows apart by their strides; draft nullable
    int64_t target_row, draft_row;
    int32_t vocab;
    const int32_t *ids;          // [n_tokens]
    const int32_t *parents;      // nullable: each token's parent is the one before it
    const int32_t *cu;
    int32_t n_seqs;
    int64_t n_tokens;
    const float *u_accept;       // [n_tokens]
    const float *u_next;         // [n_seqs]
    int32_t *n_kept, *path, *next;
};

// Where a sequence's walk stands.
struct alignas(16) Walk {
    double taken;       // what the refused drafts have taken of the node's row, in rows of the drafter's
    int32_t node;       // the last accepted token
    int32_t child;      // the child of it that was refused last (node: none yet)
    int32_t kept;       // accepted tokens
    int32_t sums;       // the round whose sums belong to this state
    int32_t over;       // no child is left: the next token is drawn
    int32_t pad[3];
};

struct VerifyPlan {
    int32_t rounds;     // launches that sum a row a sequence
    int32_t share;      // sums of a workgroup
    int32_t n_sums;     // of a row
};

struct KeepLayers {
    mrope_kv8_layer at[MROPE_MAX_LAYERS];
};

struct Keep {
    const int32_t *n_kept, *path, *cu;
    int32_t n_seqs;
    int64_t n_tokens;
    const int32_t *pos;
    int32_t n_layers, head_dim;
    Kv8 kv;             // (its caches and scales are those of the layers)
};

hipError_t launch_planes_tree(const PlanesTree &a, hipStream_t stream);
hipError_t launch_keep(const Keep &a, const KeepLayers &layers, hipStream_t stream);
VerifyPlan verify_plan(int32_t n_seqs, int32_t vocab, bool drawn_trees);
size_t verify_ws_bytes(int32_t n_seqs, const VerifyPlan &p);
hipError_t launch_verify(const Verify &a, int io, const VerifyPlan &p, void *workspace, hipStream_t stream);

}  // namespace mrope
