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

// A release's push: a bit per block of the pool in the shared memory of its blocks of
// threads, 32 warps each, a run of 32-block words per warp.
constexpr int kMaxPages = 1 << 24;               // blocks of a pool whose rows fork and are released
constexpr int kPushCtas = 16;
constexpr int kSmallBlocks = 1 << 15;            // up to as many, one block of threads pushes
constexpr int kPushMostSmem = 226 * 1024;
__host__ __device__ constexpr int push_words(int num_blocks, int ctas) {   // a warp's words
    return ((num_blocks + 31) / 32 + 32 * ctas - 1) / (32 * ctas);
}
__host__ __device__ constexpr int push_smem(int num_blocks, int ctas) { return 4 * 32 * push_words(num_blocks, ctas); }

// Its blocks of threads: one, or a cluster. Where the context has no place for a
// cluster, one for the larger pools too as far as its shared memory goes, else 0.
constexpr int push_ctas(int num_blocks, bool cluster_fits) {
    if (num_blocks <= kSmallBlocks) return 1;
    if (cluster_fits) return kPushCtas;
    return push_smem(num_blocks, 1) <= kPushMostSmem ? 1 : 0;
}

cudaError_t launch_fork(const PagesParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_release(const PagesParams &p, int num_sms, cudaStream_t st);

}  // namespace pkv
