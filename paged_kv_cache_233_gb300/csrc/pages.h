// pages.h -- parameters and launchers of the calls on a cache's pages (pages.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

struct PagesParams {
    const int32_t *choice;        // [num_seqs]: parents (fork), or lengths to keep (release)
    const int32_t *context_lens;  // [num_seqs]
    int32_t *block_tables;        // [num_seqs][max_blocks]
    int32_t *shared;              // [num_blocks]: a block's holders beyond the first
    int32_t *free_blocks;         // [free_capacity], a stack: the top is at free_count - 1
    const int32_t *free_count;    // [1]
    int32_t *block_pairs;         // fork: [num_seqs][2]
    int32_t *context_lens_out;    // [num_seqs], may be context_lens
    int32_t *free_count_out;      // [1], may be free_count
    unsigned int *err;
    int num_seqs, max_blocks, num_blocks, free_capacity, block_size;
    int shift;                    // log2(block_size), or -1
};
cudaError_t launch_fork(const PagesParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_release(const PagesParams &p, int num_sms, cudaStream_t st);

}  // namespace pkv
