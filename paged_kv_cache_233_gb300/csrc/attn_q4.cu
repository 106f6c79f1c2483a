// attn_q4.cu -- softmax attention over the 4-bit paged cache, one warp per
// (query row, kv head, up to 8 of its query heads, partition of the keys).
//
// A query row attends to the first `limit` keys of its sequence: all of them
// in decode (a row per sequence), up to its own position in prefill. A lane
// owns head_dim / 32 neighbouring channels: per key it reads their codes and
// its group's (s, m), a butterfly sums the scores over the lanes, and an online
// softmax keeps (m, l, o) per query head in fp32.
#include <cuda_runtime.h>

#include "decode_params.h"
#include "q4.cuh"

namespace pkv {

namespace {

constexpr unsigned kAllLanes = 0xffffffffu;
constexpr int kHeads = 8;      // query heads a warp serves at once
constexpr int kWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) attn_q4_kernel(const __grid_constant__ Q4AttnParams p, int rows) {
    constexpr int E = D / 32, G = D / kQ4Group;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int row = int(unit / p.max_parts), part = int(unit - (long long)row * p.max_parts);
    if (row >= rows) return;
    const int h = blockIdx.y, head0 = blockIdx.z * kHeads;
    const int g = min(kHeads, p.group - head0);
    int s = row, limit;
    if (p.query_start) {
        if (row >= __ldg(p.query_start + p.num_seqs)) return;
        int lo = 0, hi = p.num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(p.query_start + mid) <= row) lo = mid;
            else hi = mid;
        }
        s = lo;
        const int q0 = __ldg(p.query_start + s), q1 = __ldg(p.query_start + s + 1), n = q1 - q0;
        const int L = __ldg(p.context_lens + s);
        const bool rows_ok = q0 >= 0 && q1 > row && q0 <= row && q1 <= p.num_tokens && n <= p.max_query_len;
        if (!rows_ok || L < n || L > p.max_blocks * p.block_size) {
            if (lane == 0) atomicOr(p.err, rows_ok ? PAGEDKV_DEVERR_CONTEXT_LEN : PAGEDKV_DEVERR_POSITION);
            return;
        }
        limit = L - n + (row - q0) + 1;
    } else {
        const int L = __ldg(p.context_lens + s);
        limit = min(max(L, 0), p.max_blocks * p.block_size);
        if (limit != L && lane == 0) atomicOr(p.err, PAGEDKV_DEVERR_CONTEXT_LEN);
    }
    const bool split = p.part_tokens > 0 && limit > p.part_tokens;
    const int t0 = p.part_tokens > 0 ? part * p.part_tokens : 0;
    const int t1 = p.part_tokens > 0 ? min(limit, t0 + p.part_tokens) : limit;
    if (part > 0 && t0 >= limit) return;

    const T *q = reinterpret_cast<const T *>(p.q) + (size_t(row) * p.n_q_heads + h * p.group + head0) * D;
    float qf[kHeads][E], o[kHeads][E], m[kHeads], l[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
        m[j] = -INFINITY;
        l[j] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            qf[j][e] = j < g ? Elem<T>::to_float(q[j * D + lane * E + e]) * p.scale_log2 : 0.f;
            o[j][e] = 0.f;
        }
    }
    const int B = p.block_size, grp = lane * E / kQ4Group, byte = (lane * E % kQ4Group) / 2;
    for (int t = t0; t < t1; ++t) {
        int pb = __ldg(p.block_tables + size_t(s) * p.max_blocks + (t >> p.log2_block));
        if (pb < 0 || pb >= p.num_blocks) {
            if (lane == 0) atomicOr(p.err, PAGEDKV_DEVERR_BLOCK_ID);
            pb = 0;
        }
        const int off = t & (B - 1);
        const size_t base = (size_t(pb) * p.n_kv_heads + h) * q4_head_bytes(B, D);
        const size_t at = base + size_t(grp * B + off) * 16 + byte;
        const size_t pair = base + q4_pairs_at(B, D) + size_t(off * G + grp) * 4;
        float x[2][E];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const uint8_t *pool = w ? p.v_cache : p.k_cache;
            const float2 sm = q4_pair<T>(*reinterpret_cast<const uint32_t *>(pool + pair));
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = (pool[at + e / 2] >> (4 * (e & 1))) & 15;
                x[w][e] = fmaf(sm.x, float(c - 8), sm.y);
            }
        }
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            if (j >= g) break;
            float z = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) z = fmaf(qf[j][e], x[0][e], z);
#pragma unroll
            for (int mask = 16; mask >= 1; mask >>= 1) z += __shfl_xor_sync(kAllLanes, z, mask);
            const float mn = fmaxf(m[j], z);
            const float alpha = exp2f(m[j] - mn), pr = exp2f(z - mn);
            m[j] = mn;
            l[j] = fmaf(l[j], alpha, pr);
#pragma unroll
            for (int e = 0; e < E; ++e) o[j][e] = fmaf(pr, x[1][e], o[j][e] * alpha);
        }
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
        if (j >= g) break;
        const size_t qrow = size_t(row) * p.n_q_heads + h * p.group + head0 + j;
        if (split) {
            const size_t w = qrow * p.max_parts + part;
#pragma unroll
            for (int e = 0; e < E; ++e) p.ws_o[w * D + lane * E + e] = o[j][e];
            if (lane == 0) {
                p.ws_m[w] = m[j] * kLn2;
                p.ws_l[w] = l[j];
            }
        } else {
            const float inv = l[j] == 0.f ? 0.f : 1.f / l[j];
            T *out = reinterpret_cast<T *>(p.out) + qrow * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) out[e] = Elem<T>::from_float(o[j][e] * inv);
        }
    }
}

template <typename T, int D>
cudaError_t launch_typed(const Q4AttnParams &p, int rows, cudaStream_t st) {
    const long long units = (long long)rows * p.max_parts;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((units + kWarps - 1) / kWarps), unsigned(p.n_kv_heads),
                       unsigned((p.group + kHeads - 1) / kHeads));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_q4_kernel<T, D>, p, rows);
}

}  // namespace

cudaError_t launch_attn_q4(int dtype, int head_dim, const Q4AttnParams &p, int rows, cudaStream_t st) {
    if (dtype == PAGEDKV_BF16)
        return head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(p, rows, st)
                              : launch_typed<__nv_bfloat16, 128>(p, rows, st);
    return head_dim == 64 ? launch_typed<__half, 64>(p, rows, st) : launch_typed<__half, 128>(p, rows, st);
}

}  // namespace pkv
