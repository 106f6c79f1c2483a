// q8.h -- the 8-bit cache's layout and launchers, shared by host and device code.
//
// The tokens of one (block, kv head) share a scale, a power of two 2^e, and a
// channel is an e4m3 code c that stands for c * 2^e. (e4m3 has a binary exponent
// of its own: a scale that is no power of two would keep no more of a row, and a
// power of two moves the block's older codes without rounding them, but for those
// that fall below 2^-6, when a new row takes the scale up.) The bytes of one
// (block, kv head) are
//     codes  [head_dim / 16 panels][block_size tokens][16 channels]
//     scale  fp32
//     marks  32 bits, bit t set when token t's row holds a NaN; then nothing up to 16
//            bytes in all (32 in blocks of 32)
// a multiple of 16; a pool is [num_blocks][n_kv_heads] of them, so the blocks of
// neighbouring kv heads are one contiguous run that an untiled bulk copy brings in,
// scale and all. Eight tokens' codes of one panel are 128 contiguous bytes: the
// eight rows of an 8x8 matrix load without a bank conflict, in any block size.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "packed.h"

namespace pkv {

constexpr int kQ8Panel = 16;
// exponents that a scale may have: 448 * 2^120 is past bfloat16's largest value
constexpr int kQ8LeastExp = -64, kQ8MostExp = 120;

// Offset of the scale within the bytes of one (block, kv head), and their number.
__host__ __device__ constexpr int q8_scale_at(int block_size, int head_dim) { return block_size * head_dim; }
__host__ __device__ constexpr int q8_tail_bytes(int block_size) { return block_size > 16 ? block_size : 16; }
__host__ __device__ constexpr int q8_head_bytes(int block_size, int head_dim) {
    return q8_scale_at(block_size, head_dim) + q8_tail_bytes(block_size);
}

struct Q8AppendParams {
    const void *k, *v;            // [num_tokens][n_kv_heads][head_dim]
    const int32_t *block_tables;  // [num_seqs][max_blocks]
    const int32_t *query_start;   // [num_seqs + 1]
    const int32_t *context_lens;  // [num_seqs], the new rows included
    uint8_t *k_cache, *v_cache;
    unsigned int *err;
    int num_seqs, num_tokens, max_blocks, num_blocks, n_kv_heads;
    int rows;                     // rows of a CTA's tile (the launcher sets it)
};
cudaError_t launch_append_q8(const Q8AppendParams &p, int head_dim, int block_size, int dtype, int sms,
                             cudaStream_t st);
cudaError_t launch_gather_q8(const uint8_t *k_cache, const uint8_t *v_cache, const int64_t *slots, void *k,
                             void *v, int num_tokens, int n_kv_heads, int head_dim, int block_size,
                             long long num_slots, int dtype, unsigned int *err, cudaStream_t st);

// Balanced split: what a (sequence, head group) costs beside its 32-key tiles, in tiles.
constexpr int kQ8UnitCost = 2;

// Decode over the 8-bit cache, with the balanced split's merge (fixed partitions: the caller merges).
cudaError_t launch_decode_q8_f16(int head_dim, const PackedAttnParams &p, int sms, cudaStream_t st);
cudaError_t launch_decode_q8_bf16(int head_dim, const PackedAttnParams &p, int sms, cudaStream_t st);

}  // namespace pkv
