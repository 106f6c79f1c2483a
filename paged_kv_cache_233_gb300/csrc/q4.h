// q4.h -- the 4-bit cache's layout and launchers, shared by host and device code.
//
// A group is 32 neighbouring channels of one token and kv head. It has a scale
// s and a middle m, both of the cache's 16-bit type, and a channel's code c
// (0 .. 15) stands for s * (c - 8) + m. The bytes of one (block, kv head) are
//     codes  [head_dim / 32 groups][block_size tokens][16 bytes]
//            channel 2i of the group in the low half of byte i, 2i + 1 in the high half
//     pairs  [block_size tokens][head_dim / 32 groups] of (s, m)
// block_size * 5 * head_dim / 8 bytes, a multiple of 16; a pool is
// [num_blocks][n_kv_heads] of them, so the blocks of neighbouring kv heads are
// one contiguous run that an untiled bulk copy brings in. Eight tokens' codes
// of one group are 128 contiguous bytes: the eight rows of an 8x8 matrix load
// without a bank conflict, in any block size.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

constexpr int kQ4Group = 32;

// Bytes of one (block, kv head).
__host__ __device__ constexpr int q4_head_bytes(int block_size, int head_dim) {
    return block_size * head_dim * 5 / 8;
}
// Offset of the (s, m) pairs within them.
__host__ __device__ constexpr int q4_pairs_at(int block_size, int head_dim) {
    return block_size * head_dim / 2;
}

cudaError_t launch_append_q4(const void *k, const void *v, const int64_t *slots, uint8_t *k_cache,
                             uint8_t *v_cache, int num_tokens, int n_kv_heads, int head_dim,
                             int block_size, long long num_slots, int dtype,
                             unsigned int *err, cudaStream_t st);
cudaError_t launch_gather_q4(const uint8_t *k_cache, const uint8_t *v_cache, const int64_t *slots,
                             void *k, void *v, int num_tokens, int n_kv_heads, int head_dim,
                             int block_size, long long num_slots, int dtype,
                             unsigned int *err, cudaStream_t st);

struct TablesParams {
    const int32_t *new_lens;      // [num_seqs]
    const int32_t *context_lens;  // [num_seqs]
    int32_t *block_tables;        // [num_seqs][max_blocks]
    const int32_t *free_blocks;   // [free_capacity], a stack: the top is at free_count - 1
    const int32_t *free_count;    // [1]
    int32_t *query_start;         // [num_seqs + 1]
    int32_t *token_seq;           // [token_capacity]
    int32_t *token_pos;           // [token_capacity]
    int64_t *slot_mapping;        // [token_capacity] or null
    int32_t *context_lens_out;    // [num_seqs], may be context_lens
    int32_t *free_count_out;      // [1], may be free_count
    unsigned int *err;
    int num_seqs, max_blocks, free_capacity, token_capacity, block_size, num_blocks;
};
cudaError_t launch_build_tables(const TablesParams &p, int num_sms, cudaStream_t st);

// Decode over the 4-bit cache.
struct Q4AttnParams {
    const void *q;                // [num_seqs][n_q_heads][head_dim]
    const uint8_t *k_cache;
    const uint8_t *v_cache;
    const int32_t *block_tables;  // [num_seqs][max_blocks]
    const int32_t *context_lens;  // [num_seqs]
    void *out;
    float *ws_o, *ws_m, *ws_l;
    int4 *ws_cuts;                // balanced split: where pairs are cut, by pair or by CTA (decode_q4.cuh)
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

// Balanced split: what a (sequence, head group) costs beside its 32-key tiles, in tiles.
constexpr int kQ4UnitCost = 2;

// Decode, with the balanced split's merge (fixed partitions: the caller merges).
cudaError_t launch_decode_q4_f16(int head_dim, const Q4AttnParams &p, int sms, cudaStream_t st);
cudaError_t launch_decode_q4_bf16(int head_dim, const Q4AttnParams &p, int sms, cudaStream_t st);

}  // namespace pkv
