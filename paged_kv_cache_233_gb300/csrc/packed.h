// packed.h -- parameters of the decode over caches held in few bits, shared by
// host and device code.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

// Decode over a cache held in few bits (decode_packed.cuh).
struct PackedAttnParams {
    const void *q;                // [num_seqs][n_q_heads][head_dim]
    const uint8_t *k_cache;
    const uint8_t *v_cache;
    const int32_t *block_tables;  // [num_seqs][max_blocks]
    const int32_t *context_lens;  // [num_seqs]
    void *out;
    float *ws_o, *ws_m, *ws_l;
    int4 *ws_cuts;                // balanced split: where pairs are cut, by pair or by CTA
    int cuts_by_pair;
    int decode_ctas;              // the decode's grid (its launcher fills the three)
    unsigned int *err;
    float scale_log2;
    int num_seqs, n_q_heads, n_kv_heads, group;
    int num_blocks, block_size, log2_block, max_blocks;
    int part_tokens;              // tokens per partition (unsplit: the tables' whole width)
    int max_parts;
    int merged;                   // a merge kernel follows
    int balanced;                 // equal shares of the call's work per CTA, pieces joined
    int log2_hpu;                 // kv heads per unit: 4, 2 or 1
    int stages;
};

}  // namespace pkv
