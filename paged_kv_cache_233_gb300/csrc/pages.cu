// pages.cu -- sequences forked off others, and blocks given back to the free stack
// ("How a serving engine actually works", section "Copy-on-write, because you have
// used fork()"; "Paged-KV + Continuous Batching From Scratch", section 1: sharing
// a block is a count, and it is free again when its last holder lets go).
//
// shared[b] counts the holders of block b beyond the first, so that a block off
// the free stack needs no entry, whoever took it.
//
// fork: row s takes over row parents[s]'s tokens: its floor(L / B) whole blocks are
// shared (an entry copied, a count raised), and of a started block it gets a copy:
// a block off the free stack and the pair for paged_kv_copy_blocks. Children are
// granted first come, first served, as paged_kv_build_tables grants: one that needs
// a block when it is among the first free_count that do.
// release: of row s's ceil(L / B) blocks, those past the ceil(keep / B) that it keeps
// lose a holder. A count below zero marks the blocks that lost their last one: they
// go onto the stack in the order of their ids, whatever the order of the atomics.
//
// The sums over the sequences run in one block of threads, and every block runs
// them for itself; the entries are taken 32 at a time, a warp each.
#include "launch_cache.h"
#include "pages.h"
#include "ptx.cuh"
#include "scan.cuh"

namespace pkv {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kPerThread = 4;          // sequences per thread: 4096 at most

struct Divisor {                       // x / B and x % B, x >= 0
    int B, shift;
    __device__ explicit Divisor(const PagesParams &p) : B(p.block_size), shift(p.shift) {}
    __device__ int quotient(int x) const { return shift >= 0 ? x >> shift : x / B; }
    __device__ int blocks(int x) const { return quotient(x) + (x - quotient(x) * B > 0 ? 1 : 0); }   // ceil(x / B)
};

__device__ __forceinline__ int free_blocks_of(const PagesParams &p, bool report) {
    const int n = __ldcg(p.free_count);
    if (n >= 0 && n <= p.free_capacity) return n;
    if (report) atomicOr(p.err, PAGEDKV_DEVERR_POSITION);
    return min(max(n, 0), p.free_capacity);
}

// What a fork asks for s: its parent, or -1 (bad ones are reported).
__device__ __forceinline__ int parent_of(const PagesParams &p, int s, bool report) {
    const int of = __ldcg(p.choice + s);
    if (of == -1) return -1;
    if (of < 0 || of >= p.num_seqs || __ldcg(p.choice + of) != -1) {   // (a parent is no child of this call)
        if (report) atomicOr(p.err, PAGEDKV_DEVERR_SEQ_INDEX);
        return -1;
    }
    return of;
}

__device__ __forceinline__ bool bad_length(const PagesParams &p, int L) {
    return L < 0 || (long long)L > (long long)p.max_blocks * p.block_size;
}

// `totals`: write the count after the call too.
__global__ void __launch_bounds__(kMaxThreads) fork_kernel(const __grid_constant__ PagesParams p, bool totals) {
    extern __shared__ int chunk0[];    // [num_seqs + 1]: runs of 32 entries before each sequence's
    __shared__ uint2 warp_sums[32];
    const Divisor by(p);
    const int S = p.num_seqs;
    const unsigned rank = blockIdx.x;
    grid_dependency_wait();
    const int count = free_blocks_of(p, rank == 0 && threadIdx.x == 0);
    const int per = (S + int(blockDim.x) - 1) / int(blockDim.x), s0 = int(threadIdx.x) * per;
    int of[kPerThread], L[kPerThread];
    unsigned need = 0, chunks = 0, t0, t1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) of[i] = i < per && s0 + i < S ? parent_of(p, s0 + i, rank == 0) : -1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        L[i] = of[i] >= 0 ? __ldcg(p.context_lens + of[i]) : 0;
        if (bad_length(p, L[i])) {
            if (rank == 0) atomicOr(p.err, PAGEDKV_DEVERR_CONTEXT_LEN);
            of[i] = -1;
            L[i] = 0;
        }
        need += unsigned(by.blocks(L[i]) - by.quotient(L[i]));
    }
    block_scan(need, chunks, t0, t1, warp_sums);       // (no chunks yet)
    const unsigned needed = min(t0, unsigned(count));
    unsigned nth = need;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int full = by.quotient(L[i]);
        const bool started = by.blocks(L[i]) > full;
        const int s = s0 + i;
        const bool go = of[i] >= 0 && (!started || nth < unsigned(count));
        if (rank == 0 && i < per && s < S) {
            int2 pair = make_int2(0, 0);
            if (go && started) {
                const int id = __ldcg(p.free_blocks + (count - 1 - int(nth)));
                const int from = __ldcg(p.block_tables + size_t(of[i]) * p.max_blocks + full);
                if (id < 0 || id >= p.num_blocks || from < 0 || from >= p.num_blocks)
                    atomicOr(p.err, PAGEDKV_DEVERR_BLOCK_ID);
                else pair = make_int2(from, id);
                p.block_tables[size_t(s) * p.max_blocks + full] = id;
            }
            reinterpret_cast<int2 *>(p.block_pairs)[s] = pair;
            if (go) p.context_lens_out[s] = L[i];
            else if (p.context_lens_out != p.context_lens) p.context_lens_out[s] = __ldcg(p.context_lens + s);
        }
        if (started) ++nth;
        if (!go) L[i] = 0;
        chunks += unsigned(by.quotient(L[i]) + 31) / 32;
    }
    unsigned zero = 0;
    block_scan(chunks, zero, t0, t1, warp_sums);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if (i < per && s0 + i < S) {
            chunk0[s0 + i] = int(chunks);
            chunks += unsigned(by.quotient(L[i]) + 31) / 32;
        }
    }
    if (threadIdx.x == 0) chunk0[S] = int(t0);
    __syncthreads();
    if (totals && rank == 0 && threadIdx.x == 0) *p.free_count_out = count - int(needed);
    const int lane = threadIdx.x & 31, warps = int(blockDim.x >> 5);
    for (int c = int(rank) * warps + int(threadIdx.x >> 5); c < int(t0); c += int(gridDim.x) * warps) {
        const int s = last_at_or_before(chunk0, S, c);
        const int parent = __ldcg(p.choice + s);
        const int j = (c - chunk0[s]) * 32 + lane;
        if (j >= by.quotient(__ldcg(p.context_lens + parent))) continue;
        const int id = __ldcg(p.block_tables + size_t(parent) * p.max_blocks + j);
        p.block_tables[size_t(s) * p.max_blocks + j] = id;
        if (id < 0 || id >= p.num_blocks) atomicOr(p.err, PAGEDKV_DEVERR_BLOCK_ID);
        else atomicAdd(p.shared + id, 1);
    }
}

// The count after a fork, in place: how many started blocks were copied.
__global__ void __launch_bounds__(kMaxThreads) fork_total_kernel(const __grid_constant__ PagesParams p) {
    __shared__ int sums[32];
    grid_dependency_wait();
    const Divisor by(p);
    int taken = 0;
    for (int s = threadIdx.x; s < p.num_seqs; s += blockDim.x) {
        const int of = parent_of(p, s, false);
        if (of < 0) continue;
        const int L = __ldcg(p.context_lens + of);
        if (!bad_length(p, L)) taken += by.blocks(L) - by.quotient(L);
    }
    taken = __reduce_add_sync(kAllLanes, taken);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = taken;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < int(blockDim.x >> 5); ++w) taken += sums[w];
        const int count = free_blocks_of(p, false);
        *p.free_count_out = count - min(taken, count);
    }
}

// The tokens that s keeps of its L, or -1 for a bad length.
__device__ __forceinline__ int kept(const PagesParams &p, int L, int keep) {
    return bad_length(p, L) || keep < 0 ? -1 : min(L, keep);
}

__global__ void __launch_bounds__(kMaxThreads) release_kernel(const __grid_constant__ PagesParams p) {
    extern __shared__ int chunk0[];    // [num_seqs + 1]: runs of 32 entries before each sequence's
    __shared__ uint2 warp_sums[32];
    const Divisor by(p);
    const int S = p.num_seqs;
    grid_dependency_wait();
    grid_launch_dependents();
    const int per = (S + int(blockDim.x) - 1) / int(blockDim.x), s0 = int(threadIdx.x) * per;
    int given[kPerThread];
    unsigned chunks = 0, zero = 0, t0, t1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        given[i] = 0;
        if (i >= per || s0 + i >= S) continue;
        const int L = __ldcg(p.context_lens + s0 + i), keep = kept(p, L, __ldcg(p.choice + s0 + i));
        if (keep < 0) {
            if (blockIdx.x == 0) atomicOr(p.err, PAGEDKV_DEVERR_CONTEXT_LEN);
            continue;
        }
        given[i] = by.blocks(L) - by.blocks(keep);
        chunks += unsigned(given[i] + 31) / 32;
    }
    block_scan(chunks, zero, t0, t1, warp_sums);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if (i < per && s0 + i < S) {
            chunk0[s0 + i] = int(chunks);
            chunks += unsigned(given[i] + 31) / 32;
        }
    }
    if (threadIdx.x == 0) chunk0[S] = int(t0);
    __syncthreads();
    const int lane = threadIdx.x & 31, warps = int(blockDim.x >> 5);
    for (int c = int(blockIdx.x) * warps + int(threadIdx.x >> 5); c < int(t0); c += int(gridDim.x) * warps) {
        const int s = last_at_or_before(chunk0, S, c);
        const int L = __ldcg(p.context_lens + s), first = by.blocks(min(L, __ldcg(p.choice + s)));
        const int j = first + (c - chunk0[s]) * 32 + lane;
        if (j >= by.blocks(L)) continue;
        const int id = __ldcg(p.block_tables + size_t(s) * p.max_blocks + j);
        // (given back more often than it has holders: once is what it counts)
        if (id < 0 || id >= p.num_blocks || atomicSub(p.shared + id, 1) < 0) atomicOr(p.err, PAGEDKV_DEVERR_BLOCK_ID);
    }
}

// Blocks whose count went below zero, onto the stack in the order of their ids; the
// lengths and the count after the call. A cluster, a run of the blocks per warp.
constexpr int kPushCtas = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_load(const int *p, uint32_t rank) {
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

template <bool kCluster>
__global__ void __launch_bounds__(kMaxThreads) push_kernel(const __grid_constant__ PagesParams p) {
    __shared__ int warp_sums[32], total;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctas = kCluster ? kPushCtas : 1, rank = kCluster ? int(cluster_rank()) : 0;
    grid_dependency_wait();
    const int count = free_blocks_of(p, rank == 0 && threadIdx.x == 0);
    for (int s = rank * kMaxThreads + int(threadIdx.x); s < p.num_seqs; s += ctas * kMaxThreads) {
        const int L = __ldcg(p.context_lens + s), keep = kept(p, L, __ldcg(p.choice + s));
        p.context_lens_out[s] = keep < 0 ? L : keep;
    }
    // this warp's run of blocks
    const int warps = ctas * 32, per = ((p.num_blocks + warps - 1) / warps + 31) / 32 * 32;
    const int b0 = min((long long)(rank * 32 + warp) * per, (long long)p.num_blocks), b1 = min(b0 + per, p.num_blocks);
    int mine = 0;
    for (int b = b0; b < b1; b += 128) {
        int v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = b + 32 * i + lane < b1 ? __ldcg(p.shared + b + 32 * i + lane) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) mine += __popc(__ballot_sync(kAllLanes, v[i] < 0));
    }
    if (lane == 0) warp_sums[warp] = mine;
    __syncthreads();
    int w = warp_sums[lane];
    const int all = __reduce_add_sync(kAllLanes, w);
    int at = __reduce_add_sync(kAllLanes, lane < warp ? w : 0);   // pushed by the warps before this one
    int pushed = all;
    if (kCluster) {
        if (threadIdx.x == 0) total = all;
        cluster_sync();
        const int other = lane < ctas ? cluster_load(&total, uint32_t(lane)) : 0;
        at += __reduce_add_sync(kAllLanes, lane < rank ? other : 0);
        pushed = __reduce_add_sync(kAllLanes, other);
        cluster_sync();          // (no block leaves while another reads its total; every block has read the count)
    } else {
        __syncthreads();
    }
    if (rank == 0 && threadIdx.x == 0) {
        const int room = p.free_capacity - count;
        if (pushed > room) atomicOr(p.err, PAGEDKV_DEVERR_POSITION);
        *p.free_count_out = count + min(pushed, room);
    }
    if (mine == 0) return;
    at += count;
    for (int b = b0; b < b1; b += 32) {
        const bool gone = b + lane < b1 && __ldcg(p.shared + b + lane) < 0;
        const unsigned m = __ballot_sync(kAllLanes, gone);
        if (gone) {
            const int to = at + __popc(m & ((1u << lane) - 1));
            if (to < p.free_capacity) p.free_blocks[to] = b + lane;
            p.shared[b + lane] = 0;
        }
        at += __popc(m);
    }
}

cudaLaunchConfig_t config(cudaLaunchAttribute *attr, int grid, int threads, int smem, cudaStream_t st) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Threads and blocks for the sums over the sequences and a warp for each 32 entries that there may be.
void shape(const PagesParams &p, int num_sms, int &threads, int &blocks) {
    threads = 128;
    while (threads < kMaxThreads && threads * kPerThread < p.num_seqs) threads <<= 1;
    if (threads < 512 && p.num_seqs > 32) threads = 512;
    const long long warps = (long long)p.num_seqs * ((p.max_blocks + 31) / 32), want = (warps * 32 + threads - 1) / threads;
    blocks = int(want < 1 ? 1 : want < num_sms ? want : num_sms);
}

}  // namespace

cudaError_t launch_fork(const PagesParams &p, int num_sms, cudaStream_t st) {
    int threads, blocks;
    shape(p, num_sms, threads, blocks);
    const bool totals = blocks == 1 || p.free_count_out != p.free_count;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(attr, blocks, threads, int(sizeof(int)) * (p.num_seqs + 1), st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fork_kernel, p, totals);
    if (e != cudaSuccess || totals) return e;
    cfg = config(attr, 1, p.num_seqs > 256 ? kMaxThreads : 256, 0, st);
    return cudaLaunchKernelEx(&cfg, fork_total_kernel, p);
}

cudaError_t launch_release(const PagesParams &p, int num_sms, cudaStream_t st) {
    int threads, blocks;
    shape(p, num_sms, threads, blocks);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config(attr, blocks, threads, int(sizeof(int)) * (p.num_seqs + 1), st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, release_kernel, p);
    if (e != cudaSuccess) return e;
    if (p.num_blocks <= 32 * kMaxThreads) {
        cfg = config(attr, 1, kMaxThreads, 0, st);
        return cudaLaunchKernelEx(&cfg, push_kernel<false>, p);
    }
    cfg = config(attr, kPushCtas, kMaxThreads, 0, st);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kPushCtas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, push_kernel<true>, p);
}

}  // namespace pkv
