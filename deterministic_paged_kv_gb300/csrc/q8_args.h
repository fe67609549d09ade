// q8_args.h -- constants and kernel argument blocks of the 8-bit cache, shared by
// the host launch code and the kernels.  Not part of the public ABI.
#pragma once

#include "rk_internal.h"

namespace rk {

// Codes e4m3 [num_pages, Hkv, 16, D] (a page of one head is one contiguous
// 2 KiB block), scales fp32 [num_pages, Hkv], value = code * scale.  K is
// stored rotated at its token's position.
constexpr int Q8_BLOCK_BYTES = PAGE * HEAD_DIM;  // codes of one (page, KV head)
constexpr int Q8_E_MIN = -64;                    // smallest scale exponent the append writes
constexpr int Q8_E_MAX = 56;                     // largest: of inputs below 2^64 (63 - 7)
constexpr uint32_t Q8_LIMIT_BF16 = (127u + 64u) << 7;  // bf16 bit pattern of 2^64

// Build a step's tables from the rows' lengths and token counts.
struct TablesArgs {
    const int32_t* n_new;         // [B]
    const int32_t* kv_lens;       // [B], before the step
    const int32_t* pool;          // [n_pool] free page ids
    const int32_t* taken;         // [1] pages of the pool already handed out
    int32_t* block_table;         // [B, W], new entries written in place
    int32_t* kv_lens_out;         // [B] (may be kv_lens)
    int32_t* taken_out;           // [1] (may be taken)
    int32_t* qo_indptr;           // [B + 1]
    int32_t* position_ids;        // [cap]
    int32_t* slot_map;            // [cap]
    int32_t* status;
    int32_t B, W, num_pages, n_pool, cap;
};
constexpr int TAB_THREADS = 1024;
constexpr int TAB_MAX_ROWS = 16384;  // three int32 per row in shared memory

// Quantising append of n tokens.
struct AppendQ8Args {
    const void* k_new;            // bf16 [n, Hkv, D], pre-RoPE
    const void* v_new;            // bf16 [n, Hkv, D]
    const int32_t* slot_map;      // [n]: page * 16 + slot, -1 = skip
    const int32_t* position_ids;  // [n]
    uint8_t* k_cache;             // e4m3 [num_pages, Hkv, 16, D]
    uint8_t* v_cache;
    float* k_scale;               // [num_pages, Hkv]
    float* v_scale;
    int32_t* status;
    int32_t n, Hkv, num_pages;
    uint64_t rope_turns[ROPE_PAIRS];
};

// Attention over the 8-bit cache (decode: Sq = 1).
struct AttnQ8Args {
    const void* q;                // bf16 [B, Hq, Sq, D], pre-RoPE
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const float* k_scale;
    const float* v_scale;
    const int32_t* block_table;   // [B, W]
    const int32_t* kv_lens;       // [B]
    const int32_t* position_ids;  // [B, Sq]
    void* out;                    // bf16 [B, Hq, Sq, D]
    float* lse;                   // [B, Hq, Sq]
    int32_t* status;
    int32_t B, Sq, Hq, Hkv, G, W, num_pages;
    float qk_scale_log2;          // sm_scale * log2(e)
    uint32_t wait_limit_ns;
    int32_t timeout_drill;
    // decode: where a row's keys are split, zones of equal splits from a token (and split) on
    // (a second zone that is not used starts at INT32_MAX); n_splits to a row of the scratch: with
    // more than one, partial o / l [B, Hq, n_splits, D] and log2-domain LSE [B, Hq, n_splits]
    // (`step`, `steps`: where a zone starts and what a split of it takes, in steps of the kernel)
    struct {
        int32_t split, token, size, step, steps;
    } zone[2];
    int32_t n_splits;
    float* o_part;
    float* lse_part;
    uint64_t rope_turns[ROPE_PAIRS];
};

}  // namespace rk
