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
// them for itself, keeping what each sequence's entries need in shared memory; the
// entries are taken 64 at a time, a warp each with its loads in flight. The push
// is a cluster's work: a bit per block in shared memory, counts over the cluster by
// distributed shared memory, then the marked ids from the bits.
//
// Bound by launches and dependent reads (a length, an entry, a count; the entries and
// counts of the second case below are 2 us of bandwidth). Measured (one GB300, us,
// in a graph, fork, release and a copy of what they change):
//     24 + 8 rows of up to 1500 tokens            9.6
//     1024 + 1000 rows of up to 8192 tokens      25.7, of which the fork 10.1
// With runs of 128 entries 27.7, of 32 entries 27.1; before the runs, and with the push by one block of threads,
// the whole took 40 us, 28 with them (not in a graph).
#include "launch_cache.h"
#include "pages.h"
#include "ptx.cuh"
#include "scan.cuh"

namespace pkv {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kPerThread = 4;          // sequences per thread: 4096 at most
constexpr int kRun = 64;               // entries of a warp's run

struct Divisor {                       // x / B and x % B, x >= 0
    int B, shift;
    __device__ explicit Divisor(const PagesParams &p) : B(p.block_size), shift(p.shift) {}
    __device__ int quotient(int x) const { return shift >= 0 ? x >> shift : x / B; }
    __device__ int blocks(int x) const { return quotient(x) + (x - quotient(x) * B > 0 ? 1 : 0); }   // ceil(x / B)
};

// The blocks on the stack, n as it was read. (Checks come after the loads that do not
// depend on them: a kernel here is a few dependent reads long.)
__device__ __forceinline__ int free_blocks_of(const PagesParams &p, int n, bool report) {
    if (n >= 0 && n <= p.free_capacity) return n;
    if (report) atomicOr(p.err, PAGEDKV_DEVERR_POSITION);
    return min(max(n, 0), p.free_capacity);
}

__device__ __forceinline__ bool bad_length(const PagesParams &p, int L) {
    return L < 0 || (long long)L > (long long)p.max_blocks * p.block_size;
}

// What a fork asks for with parent `of`: the parent again (or -1) and its tokens. Bad ones are reported.
struct Parent {
    int above, tokens;       // its own parent, its length
    __device__ void read(const PagesParams &p, int of) {
        const bool in = of >= 0 && of < p.num_seqs;
        above = in ? __ldcg(p.choice + of) : 0;
        tokens = in ? __ldcg(p.context_lens + of) : 0;
    }
    __device__ int check(const PagesParams &p, int of, bool report, int &L) const {
        L = 0;
        if (of == -1) return -1;
        if (above != -1) {              // (a parent is no child of this call)
            if (report) atomicOr(p.err, PAGEDKV_DEVERR_SEQ_INDEX);
            return -1;
        }
        if (bad_length(p, tokens)) {
            if (report) atomicOr(p.err, PAGEDKV_DEVERR_CONTEXT_LEN);
            return -1;
        }
        L = tokens;
        return of;
    }
};

// What the entries' part of a kernel needs of each sequence, in shared memory.
struct Runs {
    int *run0;            // [num_seqs + 1]: runs before each sequence's
    int *count;           // [num_seqs]: entries
    int *from;            // [num_seqs]: the parent's row (fork), the first of them (release)
    __device__ Runs(int *memory, int S) : run0(memory), count(memory + S + 1), from(memory + 2 * S + 1) {}
};
int runs_bytes(int S) { return 4 * (3 * S + 1); }
__device__ __forceinline__ unsigned runs_of(int entries) { return unsigned(entries + kRun - 1) / kRun; }

// Every run of entries there is, a warp each: body(sequence, its first entry's number, entries left).
template <typename Body>
__device__ __forceinline__ void for_runs(const Runs &r, int S, int total, Body body) {
    const int warps = int(blockDim.x >> 5);
    for (int c = int(blockIdx.x) * warps + int(threadIdx.x >> 5); c < total; c += int(gridDim.x) * warps) {
        const int s = last_at_or_before(r.run0, S, c), first = (c - r.run0[s]) * kRun;
        body(s, first, r.count[s] - first);
    }
}

// `totals`: write the count after the call too.
__global__ void __launch_bounds__(kMaxThreads) fork_kernel(const __grid_constant__ PagesParams p, bool totals) {
    extern __shared__ int memory[];
    __shared__ uint2 warp_sums[32];
    const Divisor by(p);
    const int S = p.num_seqs;
    const Runs r(memory, S);
    const unsigned rank = blockIdx.x;
    grid_dependency_wait();
    const int on_stack = __ldcg(p.free_count);
    const int per = (S + int(blockDim.x) - 1) / int(blockDim.x), s0 = int(threadIdx.x) * per;
    int of[kPerThread], L[kPerThread];
    Parent parent[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) of[i] = i < per && s0 + i < S ? __ldcg(p.choice + s0 + i) : -1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) parent[i].read(p, of[i]);
    const int count = free_blocks_of(p, on_stack, rank == 0 && threadIdx.x == 0);
    unsigned need = 0, runs = 0, t0, t1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        of[i] = parent[i].check(p, of[i], rank == 0, L[i]);
        need += unsigned(by.blocks(L[i]) - by.quotient(L[i]));
        runs += runs_of(by.quotient(L[i]));
    }
    block_scan(need, runs, t0, t1, warp_sums);
    // A child's started block: which one it gets, and what it is a copy of. (The
    // blocks take turns with the sequences.)
    int id[kPerThread], source[kPerThread];
    unsigned nth = need, granted = 0, granted_runs = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int full = by.quotient(L[i]), s = s0 + i;
        const bool started = by.blocks(L[i]) > full;
        const bool go = of[i] >= 0 && (!started || nth < unsigned(count));
        id[i] = source[i] = 0;
        if (go && started && unsigned(s) % gridDim.x == rank) {
            id[i] = __ldcg(p.free_blocks + (count - 1 - int(nth)));
            source[i] = __ldcg(p.block_tables + size_t(of[i]) * p.max_blocks + full);
        }
        if (started) ++nth;
        if (go) {
            granted |= 1u << i;
            granted_runs += runs_of(full);
        }
    }
    const unsigned needed = min(t0, unsigned(count));
    if (t0 > unsigned(count)) {            // not all of them are granted
        unsigned zero = 0, t;
        runs = granted_runs;
        block_scan(runs, zero, t1, t, warp_sums);
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if (i < per && s0 + i < S) {
            const int entries = (granted >> i) & 1u ? by.quotient(L[i]) : 0;
            r.run0[s0 + i] = int(runs);
            r.count[s0 + i] = entries;
            r.from[s0 + i] = of[i];
            runs += runs_of(entries);
        }
    }
    if (threadIdx.x == 0) r.run0[S] = int(t1);
    __syncthreads();
    if (totals && rank == 0 && threadIdx.x == 0) *p.free_count_out = count - int(needed);
    const int lane = threadIdx.x & 31;
    for_runs(r, S, int(t1), [&](int s, int first, int left) {
        const int32_t *src = p.block_tables + size_t(r.from[s]) * p.max_blocks + first + lane;
        int32_t *dst = p.block_tables + size_t(s) * p.max_blocks + first + lane;
        int id[kRun / 32];
#pragma unroll
        for (int i = 0; i < kRun / 32; ++i) id[i] = 32 * i + lane < left ? __ldcg(src + 32 * i) : 0;
#pragma unroll
        for (int i = 0; i < kRun / 32; ++i) {
            if (32 * i + lane >= left) continue;
            dst[32 * i] = id[i];
            if (id[i] < 0 || id[i] >= p.num_blocks) atomicOr(p.err, PAGEDKV_DEVERR_BLOCK_ID);
            else atomicAdd(p.shared + id[i], 1);
        }
    });
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int s = s0 + i, full = by.quotient(L[i]);
        if (i >= per || s >= S || unsigned(s) % gridDim.x != rank) continue;
        const bool go = (granted >> i) & 1u;
        int2 pair = make_int2(0, 0);
        if (go && by.blocks(L[i]) > full) {
            if (id[i] < 0 || id[i] >= p.num_blocks || source[i] < 0 || source[i] >= p.num_blocks)
                atomicOr(p.err, PAGEDKV_DEVERR_BLOCK_ID);
            else pair = make_int2(source[i], id[i]);
            p.block_tables[size_t(s) * p.max_blocks + full] = id[i];
        }
        reinterpret_cast<int2 *>(p.block_pairs)[s] = pair;
        if (go) p.context_lens_out[s] = L[i];
        else if (p.context_lens_out != p.context_lens) p.context_lens_out[s] = __ldcg(p.context_lens + s);
    }
}

// The count after a fork, in place: how many started blocks were copied.
__global__ void __launch_bounds__(kMaxThreads) fork_total_kernel(const __grid_constant__ PagesParams p) {
    __shared__ int sums[32];
    grid_dependency_wait();
    const Divisor by(p);
    int taken = 0;
    for (int s = threadIdx.x; s < p.num_seqs; s += blockDim.x) {
        int L;
        const int of = __ldcg(p.choice + s);
        Parent parent;
        parent.read(p, of);
        parent.check(p, of, false, L);
        taken += by.blocks(L) - by.quotient(L);
    }
    taken = __reduce_add_sync(kAllLanes, taken);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = taken;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < int(blockDim.x >> 5); ++w) taken += sums[w];
        const int count = free_blocks_of(p, __ldcg(p.free_count), false);
        *p.free_count_out = count - min(taken, count);
    }
}

// The tokens that s keeps of its L, or -1 for a bad length.
__device__ __forceinline__ int kept(const PagesParams &p, int L, int keep) {
    return bad_length(p, L) || keep < 0 ? -1 : min(L, keep);
}

// The blocks that are given back lose a holder.
__device__ __forceinline__ void drop_holders(const PagesParams &p, int *memory, uint2 *warp_sums) {
    const Divisor by(p);
    const int S = p.num_seqs;
    const Runs r(memory, S);
    const int per = (S + int(blockDim.x) - 1) / int(blockDim.x), s0 = int(threadIdx.x) * per;
    int L[kPerThread], keep[kPerThread];
    unsigned runs = 0, zero = 0, t0, t1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const bool in = i < per && s0 + i < S;
        L[i] = in ? __ldcg(p.context_lens + s0 + i) : 0;
        keep[i] = in ? __ldcg(p.choice + s0 + i) : 0;
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        keep[i] = kept(p, L[i], keep[i]);
        if (keep[i] < 0) {
            if (blockIdx.x == 0) atomicOr(p.err, PAGEDKV_DEVERR_CONTEXT_LEN);
            keep[i] = L[i] = 0;
        }
        runs += runs_of(by.blocks(L[i]) - by.blocks(keep[i]));
    }
    block_scan(runs, zero, t0, t1, warp_sums);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if (i < per && s0 + i < S) {
            const int given = by.blocks(L[i]) - by.blocks(keep[i]);
            r.run0[s0 + i] = int(runs);
            r.count[s0 + i] = given;
            r.from[s0 + i] = by.blocks(keep[i]);
            runs += runs_of(given);
        }
    }
    if (threadIdx.x == 0) r.run0[S] = int(t0);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for_runs(r, S, int(t0), [&](int s, int first, int left) {
        const int32_t *src = p.block_tables + size_t(s) * p.max_blocks + r.from[s] + first + lane;
        int id[kRun / 32];
#pragma unroll
        for (int i = 0; i < kRun / 32; ++i) id[i] = 32 * i + lane < left ? __ldcg(src + 32 * i) : 0;
#pragma unroll
        for (int i = 0; i < kRun / 32; ++i) {
            // (given back more often than it has holders: once is what it counts)
            if (32 * i + lane < left && (id[i] < 0 || id[i] >= p.num_blocks || atomicSub(p.shared + id[i], 1) < 0))
                atomicOr(p.err, PAGEDKV_DEVERR_BLOCK_ID);
        }
    });
}

// Blocks whose count went below zero, onto the stack in the order of their ids; the
// lengths and the count after the call. A run of 32-block words per warp.
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
__device__ __forceinline__ void push(const PagesParams &p, uint32_t *words) {
    __shared__ int warp_sums[32], total;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctas = kCluster ? kPushCtas : 1, rank = kCluster ? int(cluster_rank()) : 0;
    const int on_stack = __ldcg(p.free_count);
    constexpr int kSeqs = kCluster ? 1 : kPerThread;         // of a thread
    int L[kSeqs], keep[kSeqs];
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        const int s = (rank * kSeqs + i) * kMaxThreads + int(threadIdx.x);
        L[i] = s < p.num_seqs ? __ldcg(p.context_lens + s) : 0;
        keep[i] = s < p.num_seqs ? __ldcg(p.choice + s) : 0;
    }
    // this warp's words: a bit for each block that is gone
    const int per = push_words(p.num_blocks, ctas), w0 = (rank * 32 + warp) * per;
    uint32_t *mine = words + warp * per;
    int gone = 0;
    constexpr int kBatch = 8;
    for (int w = 0; w < per; w += kBatch) {
        int v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const long long b = (long long)(w0 + w + i) * 32 + lane;
            v[i] = w + i < per && b < p.num_blocks ? __ldcg(p.shared + b) : 0;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const unsigned m = __ballot_sync(kAllLanes, v[i] < 0);
            gone += __popc(m);
            if (lane == 0 && w + i < per) mine[w + i] = m;
        }
    }
    if (lane == 0) warp_sums[warp] = gone;
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        const int s = (rank * kSeqs + i) * kMaxThreads + int(threadIdx.x);
        const int k = kept(p, L[i], keep[i]);
        if (s < p.num_seqs) p.context_lens_out[s] = k < 0 ? L[i] : k;
    }
    const int count = free_blocks_of(p, on_stack, rank == 0 && threadIdx.x == 0);
    __syncthreads();
    const int sum = warp_sums[lane], all = __reduce_add_sync(kAllLanes, sum);
    int at = __reduce_add_sync(kAllLanes, lane < warp ? sum : 0);   // pushed by the warps before this one
    int pushed = all;
    if (kCluster) {
        if (threadIdx.x == 0) total = all;
        cluster_sync();
        const int other = lane < ctas ? cluster_load(&total, uint32_t(lane)) : 0;
        at += __reduce_add_sync(kAllLanes, lane < rank ? other : 0);
        pushed = __reduce_add_sync(kAllLanes, other);
        cluster_sync();          // (no block leaves while another reads its total; every block has read the count)
    }
    if (rank == 0 && threadIdx.x == 0) {
        const int room = p.free_capacity - count;
        if (pushed > room) atomicOr(p.err, PAGEDKV_DEVERR_POSITION);
        *p.free_count_out = count + min(pushed, room);
    }
    if (gone == 0) return;
    at += count;
    for (int w = 0; w < per; ++w) {
        const unsigned m = mine[w];
        const int b = (w0 + w) * 32 + lane;
        if ((m >> lane) & 1u) {
            const int to = at + __popc(m & ((1u << lane) - 1));
            if (to < p.free_capacity) p.free_blocks[to] = b;
            p.shared[b] = 0;
        }
        at += __popc(m);
    }
}

__global__ void __launch_bounds__(kMaxThreads) release_kernel(const __grid_constant__ PagesParams p) {
    extern __shared__ int memory[];
    __shared__ uint2 warp_sums[32];
    grid_dependency_wait();
    grid_launch_dependents();
    drop_holders(p, memory, warp_sums);
}

template <bool kCluster>
__global__ void __launch_bounds__(kMaxThreads) push_kernel(const __grid_constant__ PagesParams p) {
    extern __shared__ int memory[];
    grid_dependency_wait();
    push<kCluster>(p, reinterpret_cast<uint32_t *>(memory));
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

// Threads and blocks for the sums over the sequences and a warp for each run of entries that there may be.
void shape(const PagesParams &p, int num_sms, int &threads, int &blocks) {
    threads = p.num_seqs > 512 ? kMaxThreads : p.num_seqs > 32 ? 512 : 128;
    const long long warps = (long long)p.num_seqs * ((p.max_blocks + kRun - 1) / kRun), want = (warps * 32 + threads - 1) / threads;
    blocks = int(want < 1 ? 1 : want < num_sms ? want : num_sms);
}

// Beyond 48 KB, static part included, a block's shared memory has to be asked for (more
// than 4000 rows or so; the question costs the host time).
template <typename Kernel>
cudaError_t open_runs(std::atomic<unsigned long long> *opened, Kernel kernel, int smem) {
    if (smem <= 47 * 1024) return cudaSuccess;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : open_dynamic_smem(opened, dev, kernel, smem);
}

}  // namespace

cudaError_t launch_fork(const PagesParams &p, int num_sms, cudaStream_t st) {
    int threads, blocks;
    shape(p, num_sms, threads, blocks);
    static std::atomic<unsigned long long> opened[kLaunchCacheDevices];
    cudaError_t e = open_runs(opened, fork_kernel, runs_bytes(p.num_seqs));
    if (e != cudaSuccess) return e;
    const bool totals = blocks == 1 || p.free_count_out != p.free_count;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(attr, blocks, threads, runs_bytes(p.num_seqs), st);
    e = cudaLaunchKernelEx(&cfg, fork_kernel, p, totals);
    if (e != cudaSuccess || totals) return e;
    cfg = config(attr, 1, p.num_seqs > 256 ? kMaxThreads : 256, 0, st);
    return cudaLaunchKernelEx(&cfg, fork_total_kernel, p);
}

cudaError_t launch_release(const PagesParams &p, int num_sms, cudaStream_t st) {
    int threads, blocks, dev = 0;
    shape(p, num_sms, threads, blocks);
    // Whatever may refuse a launch comes before the first one: holders that are taken
    // away and blocks that are not pushed would be lost.
    static std::atomic<unsigned long long> opened_runs[kLaunchCacheDevices];
    cudaError_t e = open_runs(opened_runs, release_kernel, runs_bytes(p.num_seqs));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t push;
    int ctas = 1;
    if (p.num_blocks > kSmallBlocks) {
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        static std::atomic<unsigned long long> opened[kLaunchCacheDevices];
        e = open_dynamic_smem(opened, dev, push_kernel<true>, push_smem(kMaxPages, kPushCtas));
        if (e != cudaSuccess) return e;
        push = config(attr, kPushCtas, kMaxThreads, push_smem(kMaxPages, kPushCtas), st);
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = kPushCtas;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        push.numAttrs = 2;
        // (a cluster of 16 needs as many SMs of one GPC at once: asked for the largest pool's)
        static std::atomic<unsigned long long> room[kLaunchCacheDevices];
        ctas = push_ctas(p.num_blocks, cluster_fits(room, dev, push_kernel<true>, push));
        if (ctas == 0) return cudaErrorLaunchOutOfResources;
        push.dynamicSmemBytes = size_t(push_smem(p.num_blocks, kPushCtas));
    }
    if (ctas == 1) {
        const int smem = push_smem(p.num_blocks, 1);
        static std::atomic<unsigned long long> opened[kLaunchCacheDevices];
        e = open_runs(opened, push_kernel<false>, smem);
        if (e != cudaSuccess) return e;
        push = config(attr, 1, kMaxThreads, smem, st);
    }
    cudaLaunchAttribute early[1];
    const cudaLaunchConfig_t cfg = config(early, blocks, threads, runs_bytes(p.num_seqs), st);
    e = cudaLaunchKernelEx(&cfg, release_kernel, p);
    if (e != cudaSuccess) return e;
    return ctas == 1 ? cudaLaunchKernelEx(&push, push_kernel<false>, p) : cudaLaunchKernelEx(&push, push_kernel<true>, p);
}

}  // namespace pkv
