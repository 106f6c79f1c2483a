// cache_q8.cu -- rows into the 8-bit cache and back out of it (q8.h).
//
// append: sequence s's new rows are the last n_s tokens of its context. The rows
// that fall into one block, a run, set the scale of each kv head's part of it:
//     2^e the smallest power of two (at least 2^-64) with |x| <= 448 * 2^e for
//     every finite x of the run, and no smaller than the block's scale where the
//     block holds tokens from before;
//     c = x / 2^e rounded to e4m3, ties to even; a NaN or an infinity is NaN, and
//     the token's bit is set in the block's marks.
// Where the block's older tokens had a smaller scale their codes are divided by
// the growth and rounded again. A block without older tokens starts over, so that
// what it held for another sequence never matters.
// gather: x = c * 2^e, rounded to the 16-bit type, its largest value at most.
//
// append: whoever holds a run's first row owns the run (sequence, positions and
// block follow from the offsets, so no two owners meet in a block, and nothing is
// sorted, counted or locked), and a warp takes the run of one kv head of K or V: its
// rows stay in registers between the largest value and the codes, so each is read
// once. A lane holds a panel of a row, 32 bytes in, 16 out (half a panel a lane, whole
// lines a load: 3% slower). Bound by memory latency: what counts is how many warps have
// their rows in flight, hence four CTAs to an SM where a run's rows fit 64 registers.
//
// Measured (one GB300, us; GB/s of rows in and codes out, or the other way):
//                                                       append        gather
//     64 rows of 8 heads of 128, blocks of 16            3.2           2.0
//     12 x 1024 rows, the same                          12.7 (4480)   12.4 (4650)
//         blocks of 8                                   13.1 (4350)   12.2 (4690)
//         blocks of 32                                  15.9 (3590)   12.4 (4730)
//     16,383 rows of 32 heads of 64, blocks of 32       36.6 (5500)   40.4 (4980)
//     16,383 rows of 8 heads of 128, blocks of 16       20.7 (4870)   20.3 (4980)
//         blocks of 8                                   22.0 (4570)   20.3 (4960)
//         blocks of 32                                  21.4 (4710)   20.2 (5000)
// (A run of 32 rows of 128 takes 121 registers: two CTAs to an SM, where the others have four.)
// append with three CTAs to an SM, as its registers come out by themselves: 14.8, 38.9
// and 21.5; with tiles of 16 rows, or CTAs of 128 or 512 threads: up to 20% slower.
#include <limits.h>
#include <math.h>

#include "launch_cache.h"
#include "q8.cuh"

namespace pkv {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;          // append
constexpr int kGatherThreads = 128, kGatherItems = 2;
template <int D> constexpr int gather_tokens() { return kGatherThreads * kGatherItems / (D / 8); }   // of a CTA
constexpr int kMaxTile = 32;        // rows of a CTA's tile at most: a lane each

template <typename T> constexpr uint32_t kInfBits = Elem<T>::kBf16 ? 0x7f80u : 0x7c00u;

struct Run {
    int row, count;      // its rows
    int held;            // tokens of the block before them
    int block;
};

// This lane's row t begins a run: fills it. (Bad sequences are reported by report_bad.)
__device__ __forceinline__ bool run_of(const Q8AppendParams &p, const int *starts, int t, int B, Run &x) {
    if (t >= p.num_tokens) return false;
    int lo = 0, hi = p.num_seqs;             // the last s whose first row is at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int q0 = starts[lo], q1 = starts[lo + 1], n = q1 - q0;
    if (q0 < 0 || q0 > t || q1 <= t || q1 > p.num_tokens) return false;
    const int L = __ldg(p.context_lens + lo);
    if (L < n || L > p.max_blocks * B) return false;
    const int pos = L - n + (t - q0);
    x.held = pos & (B - 1);
    if (t != q0 && x.held != 0) return false;
    x.row = t;
    x.count = min(B - x.held, q1 - t);
    x.block = __ldg(p.block_tables + size_t(lo) * p.max_blocks + pos / B);
    if (x.block < 0 || x.block >= p.num_blocks) {
        atomicOr(p.err, PAGEDKV_DEVERR_BLOCK_ID);
        return false;
    }
    return true;
}

// The checks of a prefill call's offsets and lengths, for every sequence.
__device__ __forceinline__ void report_bad(const Q8AppendParams &p, const int *starts, int B) {
    for (int s = threadIdx.x; s < p.num_seqs; s += kThreads) {
        const int q0 = starts[s], q1 = starts[s + 1], L = __ldg(p.context_lens + s);
        if (q0 < 0 || q1 < q0 || q1 > p.num_tokens) atomicOr(p.err, PAGEDKV_DEVERR_POSITION);
        else if (L < q1 - q0 || L > p.max_blocks * B) atomicOr(p.err, PAGEDKV_DEVERR_CONTEXT_LEN);
    }
}

template <typename T, int D, int B>
__global__ void __launch_bounds__(kThreads, D * B <= 2048 ? 4 : 2) append_q8_kernel(const __grid_constant__ Q8AppendParams p) {
    constexpr int kPanels = D / kQ8Panel;
    constexpr int kRows = 32 / kPanels;                 // rows of a pass
    constexpr int kPasses = B > kRows ? B / kRows : 1;
    extern __shared__ int starts[];                     // [num_seqs + 1]
    __shared__ Run runs[kMaxTile];
    __shared__ int num_runs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // every input may come from the kernel before this one; only then may the
    // kernel after this one start
    grid_dependency_wait();
    grid_launch_dependents();
    for (int s = threadIdx.x; s <= p.num_seqs; s += kThreads) starts[s] = __ldg(p.query_start + s);
    __syncthreads();
    if (warp == 0) {
        Run x;
        const bool mine = lane < p.rows && run_of(p, starts, int(blockIdx.x) * p.rows + lane, B, x);
        const unsigned m = __ballot_sync(kAll, mine);
        if (mine) runs[__popc(m & ((1u << lane) - 1))] = x;
        if (lane == 0) num_runs = __popc(m);
    }
    __syncthreads();
    const int H = p.n_kv_heads;
    const int panel = lane % kPanels, r0 = lane / kPanels;
    const int o = blockIdx.y;
    const uint4 *src = static_cast<const uint4 *>(o ? p.v : p.k);
    uint8_t *pool = o ? p.v_cache : p.k_cache;
    for (int u = warp; u < num_runs * H; u += kThreads / 32) {
        const Run x = runs[u / H];
        const int h = u % H;
        uint8_t *base = pool + (size_t(x.block) * H + h) * q8_head_bytes(B, D);
        float *scale_at = reinterpret_cast<float *>(base + q8_scale_at(B, D));
        uint4 w[kPasses][2];
        uint32_t top2 = 0;
        const uint2 was = x.held ? *reinterpret_cast<const uint2 *>(scale_at) : make_uint2(0u, 0u);
        uint32_t marks = was.y & ((1ull << x.held) - 1);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = i * kRows + r0;
            w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
            if (r < x.count) {
                const uint4 *a = src + ((size_t(x.row) + r) * H + h) * (D / 8) + panel * 2;
                w[i][0] = __ldcs(a);
                w[i][1] = __ldcs(a + 1);
            }
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint4 v = w[i][j];
                top2 = __vmaxu2(__vmaxu2(top2, v.x & 0x7fff7fffu), __vmaxu2(v.y & 0x7fff7fffu, v.z & 0x7fff7fffu));
                top2 = __vmaxu2(top2, v.w & 0x7fff7fffu);
            }
        }
        uint32_t top = __reduce_max_sync(kAll, max(top2 & 0xffffu, top2 >> 16));
        if (top >= kInfBits<T>) {
            // a NaN or an infinity among them: each becomes a NaN, and the others set the scale
            top = 0;
            uint32_t mine = 0;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t c[4] = {w[i][j].x, w[i][j].y, w[i][j].z, w[i][j].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t lo = c[e] & 0x7fffu, hi = (c[e] >> 16) & 0x7fffu;
                        if (lo >= kInfBits<T>) c[e] |= 0x7fffu;
                        else top = max(top, lo);
                        if (hi >= kInfBits<T>) c[e] |= 0x7fff0000u;
                        else top = max(top, hi);
                        if (max(lo, hi) >= kInfBits<T>) mine |= 1u << ((i * kRows + r0) & 31);
                    }
                    w[i][j] = make_uint4(c[0], c[1], c[2], c[3]);
                }
            }
            top = __reduce_max_sync(kAll, top);
            marks |= __reduce_or_sync(kAll, mine) << x.held;
        }
        int e = q8_exponent_for(Elem<T>::unpack2(top).x);
        const int before = x.held ? min(max(q8_exponent(__uint_as_float(was.x)), kQ8LeastExp), kQ8MostExp) : e;
        if (before < e) {
            // the block's older codes under the larger scale (a result below 2^-10 is zero)
            const float shrink = q8_power(max(before - e, -100));
            for (int y = lane; y < x.held * kPanels; y += 32) {
                uint4 *at = reinterpret_cast<uint4 *>(base + (y / x.held) * B * 16) + y % x.held;
                const uint4 v = *at;
                auto smaller = [&](uint32_t c) {
                    uint32_t lo, hi;
                    q8_halves(c, lo, hi);
                    const float2 a = Elem<__half>::unpack2(lo), b = Elem<__half>::unpack2(hi);
                    return q8_codes(a.x * shrink, a.y * shrink, b.x * shrink, b.y * shrink);
                };
                *at = make_uint4(smaller(v.x), smaller(v.y), smaller(v.z), smaller(v.w));
            }
        }
        e = max(e, before);
        const float inv = q8_power(-e);
        auto four = [&](uint32_t a, uint32_t b) {
            const float2 x = Elem<T>::unpack2(a), y = Elem<T>::unpack2(b);
            return q8_codes(x.x * inv, x.y * inv, y.x * inv, y.y * inv);
        };
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = i * kRows + r0;
            if (r < x.count) {
                const uint4 a = w[i][0], b = w[i][1];
                *reinterpret_cast<uint4 *>(base + (panel * B + x.held + r) * 16) =
                    make_uint4(four(a.x, a.y), four(a.z, a.w), four(b.x, b.y), four(b.z, b.w));
            }
        }
        if (lane == 0) *reinterpret_cast<uint2 *>(scale_at) = make_uint2(__float_as_uint(q8_power(e)), marks);
    }
    if (blockIdx.x == 0 && o == 0) report_bad(p, starts, B);
}

struct GatherParams {
    const int64_t *slots;
    const uint8_t *cache[2];      // K, V
    uint4 *rows[2];               // k, v [num_tokens][n_kv_heads][head_dim]
    unsigned int *err;
    int num_tokens, n_kv_heads, log2_block;
    long long num_slots;
};

// An item is half a panel of a token: 8 bytes in, 16 out. A CTA takes some tokens of
// one kv head of K or V, four neighbouring tokens' half panels as neighbouring items:
// whole sectors where their slots are neighbours, as a prompt's are. Its issue slots are
// two thirds used: heads by blockIdx and the products packed where they can be (fp16)
// took 12 x 1024 rows from 13.0 to 12.4 us.
template <typename T, int D>
__global__ void __launch_bounds__(kGatherThreads) gather_q8_kernel(const __grid_constant__ GatherParams p) {
    // (no early start for the kernel after this one: its work, rows of these to
    // append or attend over, comes after this grid's end)
    grid_dependency_wait();
    constexpr int kHalves = D / 8, kTokens = gather_tokens<D>();
    constexpr float kMost = Elem<T>::kBf16 ? 0x1.fep127f : 65504.f;
    const int o = blockIdx.y, B = 1 << p.log2_block;
    const int tile = blockIdx.x / unsigned(p.n_kv_heads), h = blockIdx.x - tile * p.n_kv_heads;
    const uint8_t *pool = p.cache[o] + size_t(h) * q8_head_bytes(B, D);
    const size_t block_bytes = size_t(p.n_kv_heads) * q8_head_bytes(B, D);
    const int half = threadIdx.x & 1;
    long long slot[kGatherItems];
    int token[kGatherItems], panel[kGatherItems];
#pragma unroll
    for (int i = 0; i < kGatherItems; ++i) {
        const int x = (int(threadIdx.x) + i * kGatherThreads) >> 1;       // [quad][panel][4 tokens]
        panel[i] = (x >> 2) % (kHalves / 2);
        token[i] = tile * kTokens + (x >> 2) / (kHalves / 2) * 4 + (x & 3);
        slot[i] = token[i] < p.num_tokens ? __ldg(reinterpret_cast<const long long *>(p.slots) + token[i]) : -1;
        if (slot[i] >= p.num_slots) {
            if (h + panel[i] + half == 0) atomicOr(p.err, PAGEDKV_DEVERR_SLOT_RANGE);
            slot[i] = -1;
        }
    }
    uint2 c[kGatherItems];
    float scale[kGatherItems];
#pragma unroll
    for (int i = 0; i < kGatherItems; ++i) {
        if (slot[i] < 0) continue;
        const uint8_t *base = pool + size_t(slot[i] >> p.log2_block) * block_bytes;
        c[i] = *reinterpret_cast<const uint2 *>(base + (panel[i] * B + int(slot[i] & (B - 1))) * 16 + half * 8);
        scale[i] = *reinterpret_cast<const float *>(base + q8_scale_at(B, D));
    }
#pragma unroll
    for (int i = 0; i < kGatherItems; ++i) {
        if (slot[i] < 0) continue;
        uint32_t r[4];
        q8_halves(c[i].x, r[0], r[1]);
        q8_halves(c[i].y, r[2], r[3]);
        // a scale of 2^-14 .. 2^7 takes a code to fp16 in one rounding and to no
        // infinity; the others, and bf16, go through fp32
        if (!Elem<T>::kBf16 && scale[i] >= 0x1p-14f && scale[i] <= 0x1p7f) {
            const uint32_t by = pack_half2(scale[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = hmul2_u(r[j], by);
        } else {
            const bool near = fabsf(scale[i]) < (Elem<T>::kBf16 ? 0x1p119f : 0x1p7f);     // nothing past the type's range
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 f = Elem<__half>::unpack2(r[j]);
                f.x *= scale[i];
                f.y *= scale[i];
                if (!near) {      // (a NaN stays one)
                    if (fabsf(f.x) > kMost) f.x = copysignf(kMost, f.x);
                    if (fabsf(f.y) > kMost) f.y = copysignf(kMost, f.y);
                }
                r[j] = Elem<T>::pack2(f.x, f.y);
            }
        }
        __stcs(p.rows[o] + (size_t(token[i]) * p.n_kv_heads + h) * kHalves + panel[i] * 2 + half, make_uint4(r[0], r[1], r[2], r[3]));
    }
}

cudaLaunchConfig_t config(cudaLaunchAttribute *attr, dim3 grid, int threads, int smem, cudaStream_t st) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <typename T, int D, int B>
cudaError_t append_sized(Q8AppendParams p, int sms, cudaStream_t st) {
    // rows of a tile: as many as leave each SM a CTA for K and one for V
    p.rows = kMaxTile;
    while (p.rows > 1 && (long long)p.num_tokens < (long long)p.rows * sms) p.rows >>= 1;
    const dim3 grid(unsigned((p.num_tokens + p.rows - 1) / p.rows), 2);
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(&attr, grid, kThreads, int(sizeof(int)) * (p.num_seqs + 1), st);
    return cudaLaunchKernelEx(&cfg, append_q8_kernel<T, D, B>, p);
}

template <typename T>
cudaError_t append_typed(const Q8AppendParams &p, int head_dim, int block_size, int sms, cudaStream_t st) {
    if (head_dim == 64)
        return block_size == 8    ? append_sized<T, 64, 8>(p, sms, st)
               : block_size == 16 ? append_sized<T, 64, 16>(p, sms, st)
                                  : append_sized<T, 64, 32>(p, sms, st);
    return block_size == 8    ? append_sized<T, 128, 8>(p, sms, st)
           : block_size == 16 ? append_sized<T, 128, 16>(p, sms, st)
                              : append_sized<T, 128, 32>(p, sms, st);
}

template <typename T, int D>
cudaError_t gather_typed(const GatherParams &p, cudaStream_t st) {
    const long long ctas = ((long long)p.num_tokens + gather_tokens<D>() - 1) / gather_tokens<D>() * p.n_kv_heads;
    if (ctas > INT_MAX) return cudaErrorInvalidConfiguration;      // (rows of 16 TB)
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(&attr, dim3(unsigned(ctas), 2), kGatherThreads, 0, st);
    return cudaLaunchKernelEx(&cfg, gather_q8_kernel<T, D>, p);
}

}  // namespace

cudaError_t launch_append_q8(const Q8AppendParams &p, int head_dim, int block_size, int dtype, int sms,
                             cudaStream_t st) {
    return dtype == PAGEDKV_BF16 ? append_typed<__nv_bfloat16>(p, head_dim, block_size, sms, st)
                                 : append_typed<__half>(p, head_dim, block_size, sms, st);
}

cudaError_t launch_gather_q8(const uint8_t *k_cache, const uint8_t *v_cache, const int64_t *slots, void *k,
                             void *v, int num_tokens, int n_kv_heads, int head_dim, int block_size,
                             long long num_slots, int dtype, unsigned int *err, cudaStream_t st) {
    GatherParams p{};
    p.slots = slots;
    p.cache[0] = k_cache;
    p.cache[1] = v_cache;
    p.rows[0] = static_cast<uint4 *>(k);
    p.rows[1] = static_cast<uint4 *>(v);
    p.err = err;
    p.num_tokens = num_tokens;
    p.n_kv_heads = n_kv_heads;
    while ((1 << p.log2_block) < block_size) ++p.log2_block;
    p.num_slots = num_slots;
    if (dtype == PAGEDKV_BF16)
        return head_dim == 64 ? gather_typed<__nv_bfloat16, 64>(p, st)
                              : gather_typed<__nv_bfloat16, 128>(p, st);
    return head_dim == 64 ? gather_typed<__half, 64>(p, st)
                          : gather_typed<__half, 128>(p, st);
}

}  // namespace pkv
