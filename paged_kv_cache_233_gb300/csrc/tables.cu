// tables.cu -- a step's block tables, token lists and slots from the requests'
// lengths ("How a serving engine actually works", sections "The one formula"
// and "Three allocators, one workload": a sequence holds ceil(length / B)
// blocks and grows a block at a time from a free list).
//
// Request s holds c_s tokens in ceil(c_s / B) blocks and asks for n_s more,
// which opens ceil((c_s + n_s) / B) - ceil(c_s / B) blocks. Requests are
// granted first come, first served: s is granted when the blocks that requests
// 0 .. s ask for are free (or it opens none) and their tokens fit the token
// lists. A second prefix sum over the granted ones places their tokens and
// their blocks, which come off the top of the free stack.
//
// The sums run over the whole call in one block of threads, and every block
// runs them for itself, then takes its part of the tokens and the opened
// blocks. One launch, unless several blocks read lengths or a count that are
// updated in place: those are then written by a second one.
//
// Bound by latency: a launch, the lengths, a table entry or a free block. 256
// requests of a token each: 3.3 us; 2048 requests, 67,000 tokens: 6.8 us, in
// place 8.6 (by a cluster of blocks over distributed shared memory 12.6).
#include "launch_cache.h"
#include "ptx.cuh"
#include "q4.h"

namespace pkv {

namespace {

constexpr unsigned kAllLanes = 0xffffffffu;
constexpr int kMaxThreads = 1024;
constexpr int kPerThread = 4;          // requests per thread: 4096 requests at most
constexpr unsigned kFull30 = 1u << 30; // sums saturate here: past every capacity

__device__ __forceinline__ unsigned add_sat(unsigned a, unsigned b) { return min(a + b, kFull30); }

// Exclusive prefix sums of (a, b) over the block's threads, and their totals.
__device__ __forceinline__ void block_scan(unsigned &a, unsigned &b, unsigned &ta, unsigned &tb,
                                           uint2 *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
    unsigned x = a, y = b;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned u = __shfl_up_sync(kAllLanes, x, d), v = __shfl_up_sync(kAllLanes, y, d);
        if (lane >= d) {
            x = add_sat(x, u);
            y = add_sat(y, v);
        }
    }
    unsigned ex = __shfl_up_sync(kAllLanes, x, 1), ey = __shfl_up_sync(kAllLanes, y, 1);
    if (lane == 0) ex = ey = 0;
    if (lane == 31) warp_sums[warp] = make_uint2(x, y);
    __syncthreads();
    // every warp sums the warps before it, and all of them
    uint2 w = lane < warps ? warp_sums[lane] : make_uint2(0, 0);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned u = __shfl_up_sync(kAllLanes, w.x, d), v = __shfl_up_sync(kAllLanes, w.y, d);
        if (lane >= d) {
            w.x = add_sat(w.x, u);
            w.y = add_sat(w.y, v);
        }
    }
    const unsigned bx = __shfl_sync(kAllLanes, w.x, warp > 0 ? warp - 1 : 0);
    const unsigned by = __shfl_sync(kAllLanes, w.y, warp > 0 ? warp - 1 : 0);
    ta = __shfl_sync(kAllLanes, w.x, 31);
    tb = __shfl_sync(kAllLanes, w.y, 31);
    a = add_sat(ex, warp > 0 ? bx : 0);
    b = add_sat(ey, warp > 0 ? by : 0);
    __syncthreads();
}

// The last s of [0, n) whose start[s] <= x (start is non-decreasing, start[0] <= x).
__device__ __forceinline__ int last_at_or_before(const int *start, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// `totals`: write the lengths and the count after the step too.
__global__ void __launch_bounds__(kMaxThreads) build_tables_kernel(const __grid_constant__ TablesParams p, bool totals) {
    // [S + 1] each: first token, first opened block; then tokens held
    extern __shared__ int arrays[];
    __shared__ uint2 warp_sums[32];
    const int S = p.num_seqs, B = p.block_size;
    // x / B (x >= 0): a shift where B is a power of two
    const int shift = (B & (B - 1)) == 0 ? 31 - __clz(B) : -1;
    auto divide = [&](int x) { return shift >= 0 ? x >> shift : x / B; };
    int *tok0 = arrays, *blk0 = arrays + S + 1, *held_tokens = blk0 + S + 1;
    const unsigned rank = blockIdx.x, blocks = gridDim.x;
    // lengths, tables and the free stack as the kernels before this one left
    // them, and those kernels done with what is written here
    grid_dependency_wait();

    int free_count = __ldcg(p.free_count);
    if (free_count < 0 || free_count > p.free_capacity) {
        if (rank == 0 && threadIdx.x == 0) atomicOr(p.err, PAGEDKV_DEVERR_POSITION);
        free_count = min(max(free_count, 0), p.free_capacity);
    }
    // this thread's requests: `per` neighbouring ones
    const int per = (S + int(blockDim.x) - 1) / int(blockDim.x);
    const int s0 = int(threadIdx.x) * per;
    int c[kPerThread], n[kPerThread], need[kPerThread];
    unsigned a = 0, b = 0, ta, tb;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        c[i] = n[i] = need[i] = 0;
        if (i < per && s0 + i < S) {
            c[i] = __ldcg(p.context_lens + s0 + i);
            n[i] = __ldcg(p.new_lens + s0 + i);
        }
    }
    bool ok[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        ok[i] = i < per && s0 + i < S;
        if (!ok[i]) continue;
        const long long after = (long long)c[i] + n[i];
        const bool lens = c[i] >= 0 && n[i] >= 0;
        if (!lens || after > (long long)p.max_blocks * B) {
            if (rank == 0) atomicOr(p.err, lens ? PAGEDKV_DEVERR_POSITION : PAGEDKV_DEVERR_CONTEXT_LEN);
            ok[i] = false;
            continue;
        }
        need[i] = int((after + B - 1) / B) - (c[i] + B - 1) / B;
        a = add_sat(a, unsigned(need[i]));
        b = add_sat(b, unsigned(n[i]));
    }
    block_scan(a, b, ta, tb, warp_sums);
    // granted requests, and the second sums over them
    unsigned ra = a, rb = b, ga = 0, gb = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if (!ok[i]) {
            n[i] = need[i] = 0;
            continue;
        }
        ra = add_sat(ra, unsigned(need[i]));
        rb = add_sat(rb, unsigned(n[i]));
        ok[i] = (need[i] == 0 || ra <= unsigned(free_count)) && (n[i] == 0 || rb <= unsigned(p.token_capacity));
        if (!ok[i]) n[i] = need[i] = 0;
        ga += unsigned(need[i]);
        gb += unsigned(n[i]);
    }
    if (ta > unsigned(free_count) || tb > unsigned(p.token_capacity)) {   // (the same for every thread)
        a = ga;
        b = gb;
        block_scan(a, b, ta, tb, warp_sums);
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if (i < per && s0 + i < S) {
            tok0[s0 + i] = int(b);
            blk0[s0 + i] = int(a);
            held_tokens[s0 + i] = c[i];
            b += unsigned(n[i]);
            a += unsigned(need[i]);
        }
    }
    const int tokens = int(tb), opened = int(ta);
    if (threadIdx.x == 0) {
        tok0[S] = tokens;
        blk0[S] = opened;
    }
    // this block's arrays are complete, and (a single one) it has read the
    // lengths and the count that it may now overwrite
    __syncthreads();

    if (rank == 0) {
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            if (i < per && s0 + i < S) {
                if (totals) p.context_lens_out[s0 + i] = c[i] + n[i];
                p.query_start[s0 + i] = tok0[s0 + i];
            }
        }
        if (threadIdx.x == 0) {
            p.query_start[S] = tokens;
            if (totals) *p.free_count_out = free_count - opened;
        }
    }
    const int stride = int(blocks * blockDim.x);
    const int first = int(rank * blockDim.x + threadIdx.x);
    for (int x = first; x < opened; x += stride) {
        const int s = last_at_or_before(blk0, S, x);
        const int id = __ldcg(p.free_blocks + (free_count - 1 - x));
        if (id < 0 || id >= p.num_blocks) atomicOr(p.err, PAGEDKV_DEVERR_BLOCK_ID);
        p.block_tables[size_t(s) * p.max_blocks + divide(held_tokens[s] + B - 1) + (x - blk0[s])] = id;
    }
    for (int t = first; t < p.token_capacity; t += stride) {
        int s = 0, pos = -1;
        long long slot = -1;
        if (t < tokens) {
            s = last_at_or_before(tok0, S, t);
            const int held = held_tokens[s];
            pos = held + (t - tok0[s]);
            const int j = divide(pos);
            const int nth = j - divide(held + B - 1);   // which of the request's opened blocks, if any
            const int id = nth < 0 ? __ldcg(p.block_tables + size_t(s) * p.max_blocks + j)
                                   : __ldcg(p.free_blocks + (free_count - 1 - (blk0[s] + nth)));
            if (id < 0 || id >= p.num_blocks) atomicOr(p.err, PAGEDKV_DEVERR_BLOCK_ID);
            else slot = (long long)id * B + (pos - j * B);
        }
        p.token_seq[t] = s;
        p.token_pos[t] = pos;
        if (p.slot_mapping) p.slot_mapping[t] = slot;
    }
    // (No early start for the kernel after this one: what it reads of these is
    // there after its dependency wait, not before. 3.3 us a call; with an early
    // start behind a fence over every write 4.0.)
}

// The lengths and the count after a step, in place: query_start holds what each
// request was granted.
__global__ void __launch_bounds__(kMaxThreads) tables_totals_kernel(const __grid_constant__ TablesParams p) {
    __shared__ int sums[32];
    grid_dependency_wait();
    const int B = p.block_size;
    int opened = 0;
    for (int s = threadIdx.x; s < p.num_seqs; s += blockDim.x) {
        const int c = __ldcg(p.context_lens + s);
        const int n = __ldcg(p.query_start + s + 1) - __ldcg(p.query_start + s);
        p.context_lens_out[s] = c + n;
        if (n > 0) opened += int(((long long)c + n + B - 1) / B) - (c + B - 1) / B;
    }
    opened = __reduce_add_sync(kAllLanes, opened);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = opened;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < int(blockDim.x >> 5); ++w) opened += sums[w];
        *p.free_count_out = min(max(__ldcg(p.free_count), 0), p.free_capacity) - opened;
    }
}

}  // namespace

cudaError_t launch_build_tables(const TablesParams &p, int num_sms, cudaStream_t st) {
    // a token per thread, up to a block per SM
    const long long work = p.token_capacity > p.num_seqs ? p.token_capacity : p.num_seqs;
    int threads = 128;
    while (threads < kMaxThreads && (threads < work || threads * kPerThread < p.num_seqs)) threads <<= 1;
    const long long want = (work + threads - 1) / threads;
    const int blocks = want < 1 ? 1 : int(want < num_sms ? want : num_sms);
    const bool in_place = p.context_lens_out == p.context_lens || p.free_count_out == p.free_count;
    const bool totals = blocks == 1 || !in_place;
    const int smem = int(sizeof(int)) * (3 * p.num_seqs + 2);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<unsigned long long> opened[kLaunchCacheDevices];
    if (smem > 40 * 1024) {
        e = open_dynamic_smem(opened, dev, build_tables_kernel, smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, build_tables_kernel, p, totals);
    if (e != cudaSuccess || totals) return e;
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(p.num_seqs > 256 ? kMaxThreads : 256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, tables_totals_kernel, p);
}

}  // namespace pkv
