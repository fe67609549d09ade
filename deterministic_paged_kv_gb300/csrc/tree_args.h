// tree_args.h -- kernel argument blocks of the speculative step, shared by the host
// launch code and the kernels.  Not part of the public ABI.
#pragma once

#include "rk_internal.h"

namespace rk {

constexpr int TREE_MAX = 64;       // nodes of a row's tree
constexpr int TREE_UNUSED = -2;    // parent of a node that the row does not have

// Attention of the T nodes behind each row's prefix.
struct TreeArgs {
    const void* q;                // bf16 [B, Hq, T, D], pre-RoPE
    const int32_t* block_table;   // [B, W]
    const int32_t* kv_lens;       // [B], nodes included
    const int32_t* parents;       // [B, T]
    void* out;                    // bf16 [B, Hq, T, D]
    float* lse;                   // [B, Hq, T]
    int32_t* status;
    int32_t B, T, Hq, Hkv, G, W, num_pages;
    float qk_scale_log2;          // sm_scale * log2(e)
    uint32_t wait_limit_ns;
    int32_t timeout_drill;
    // where a row's prefix is cut: zones of equal parts from a token (and part) on; with more than one part to
    // the widest row: partial O / l [B, Hq, T, n_splits, D] and log2-domain LSE [B, Hq, T, n_splits]
    struct Zone {
        int32_t split, token, shift;  // parts of 2^shift tokens
    } zone[2];
    int32_t members;              // runs that a head's items are dealt to (set at the launch)
    uint64_t share;               // 2^32 / members, rounded up (set at the launch)
    int32_t n_splits;
    float* o_part;
    float* lse_part;
    uint64_t rope_turns[ROPE_PAIRS];
};

// The walk down each row's tree.
struct VerifyArgs {
    const void* logits;           // bf16 or fp32 [B, T, V]
    const float* draft_probs;     // [B, T, V] or null
    const int32_t* draft_tokens;  // [B, T]
    const int32_t* parents;       // [B, T]
    const float* coins;           // [B, T]
    const float* race;            // [B, V]
    const float* temperature;     // [B]
    int32_t* n_accepted;          // [B]
    int32_t* n_drop;              // [B]
    int32_t* path;                // [B, T]
    int32_t* tokens;              // [B, T]
    float* logprobs;              // [B, T]
    int32_t* status;
    int32_t B, T, V, f32;
    int32_t cluster;              // CTAs of a row, a power of two up to 16 (set at the launch)
};

// Accepted nodes' K and V to the slots behind the prefix.
struct CompactArgs {
    const int32_t* path;          // [B, T]
    const int32_t* n_keep;        // [B]
    const int32_t* block_table;   // [B, W]
    const int32_t* kv_lens;       // [B], nodes included
    void* k_cache;                // bf16 [num_pages, 16, Hkv, D]
    void* v_cache;
    int32_t* status;
    int32_t B, T, Hkv, W, num_pages;
};

// Which rows have a tree: those that got its T tokens.
struct TreeRowsArgs {
    const int32_t* qo_indptr;     // [B + 1]
    const int32_t* kv_lens;       // [B], nodes included
    const int32_t* parents;       // [B, T]
    int32_t* tree_lens;           // [B]
    int32_t* tree_parents;        // [B, T] (may be parents)
    int32_t* status;
    int32_t B, T;
};

// Dropped tokens' lengths and pages.
struct TrimArgs {
    const int32_t* n_drop;        // [B]
    const int32_t* kv_lens;       // [B], before the drop
    int32_t* pool;                // [n_pool]
    const int32_t* taken;         // [1]
    int32_t* block_table;         // [B, W]
    int32_t* kv_lens_out;         // [B] (may be kv_lens)
    int32_t* taken_out;           // [1] (may be taken)
    int32_t* status;
    int32_t B, W, num_pages, n_pool;
};

}  // namespace rk
