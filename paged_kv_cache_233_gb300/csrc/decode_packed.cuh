// decode_packed.cuh -- the paged-attention decode over caches held in few bits:
// units, copies, shares and merges, around a consumer that computes a tile
// (decode_q4.cuh, decode_q8.cuh).
//
// A consumer C is one warp's state for a unit's kv head: its element type, head
// size and block size, kHead bytes of a (block, kv head), CTAs per SM, what a unit
// costs beside its tiles; begin (the queries), tile (32 keys of K and V in shared
// memory), finish, and rows out of put_state and put_out. Its reference ref, in
// base 2, and its sums l go with the rows.
//
// Work. A unit is (sequence, group of H kv heads, range of keys), split whole,
// in fixed partitions or in equal shares of the call's work per CTA: its 32-key
// tiles, and a few tiles' worth (C::kUnitCost) for each (sequence, head group),
// whose queries, sums and stores cost about that. (Counting tiles alone, the
// CTAs that got many short sequences ended last: 64 sequences of 1 to 2048
// tokens, 32 heads of 64, 45.7 us against 42.4, 256 of 1 to 512 59.1 against
// 48.3; with one tile's worth 42.3 and 51.6, with three 43.4 and 50.1.)
// Per CTA one producer warp copies each tile's blocks with untiled bulk copies
// (a block's bytes of neighbouring kv heads are one run), through a ring of
// stages; four consumer warps own a kv head each (H = 4) or share one (H = 2,
// 1: every (4/H)-th tile each, joined at the unit's end). The copies mark their
// lines to be evicted first, which gains 1 to 7% past the L2's size and leaves
// smaller caches and shared prefixes at the time they had: their lines stay as
// long as nothing needs the room.
//
#pragma once

#include "decode_params.h"
#include "launch_cache.h"
#include "packed.h"
#include "ptx.cuh"

namespace pkv {

constexpr int kPackedTile = 32;            // keys per stage
constexpr int kPackedConsumers = 4;
constexpr int kPackedThreads = 32 * (1 + kPackedConsumers);
constexpr unsigned kPackedAll = 0xffffffffu;

// Balanced split: the CTAs that get a share of `total` positions (tiles and unit
// costs), none of them empty, and share c's first position.
__device__ __forceinline__ int packed_sharers(int total, int grid) { return max(1, min(grid, total)); }
__device__ __forceinline__ int packed_share(int total, int c, int sharers) {
    return int((long long)total * c / sharers);
}

// The share that holds position t.
__device__ __forceinline__ int packed_share_of(int total, int t, int sharers) {
    int c = int((long long)t * sharers / total);
    while (c + 1 < sharers && packed_share(total, c + 1, sharers) <= t) ++c;
    while (c > 0 && packed_share(total, c, sharers) > t) --c;
    return c;
}

struct PackedSmem {
    int stage_bytes, stages, seqs, head_dim, shared_heads;   // shared_heads: warps of one kv head join states
    __host__ __device__ int bars() const { return stages * stage_bytes; }
    __host__ __device__ int flag() const { return bars() + 16 * stages; }
    __host__ __device__ int scan() const { return flag() + 16; }                 // a word per warp
    __host__ __device__ int base() const { return scan() + 32; }                 // seqs + 1
    __host__ __device__ int len() const { return base() + 4 * (seqs + 1); }      // seqs
    __host__ __device__ int join() const { return (len() + 4 * seqs + 15) & ~15; }
    __host__ __device__ int row() const { return head_dim + 4; }                 // floats of a joined row
    __host__ __device__ int total() const {
        return join() + (shared_heads ? kPackedConsumers * 8 * (row() + 2) * 4 : 0);
    }
};

struct PackedUnit {
    int s, hg, t0, t1;
    int part;         // its partition; balanced split: its piece slot of the CTA
    bool partial;     // the result is a state for the merge
    int last;         // balanced split: the position of the pair's last tile where this CTA has its first, else -1
};

// This CTA's units in order; the producer and every consumer warp walk a copy.
// kUnitCost: what a (sequence, head group) costs beside its tiles, in tiles.
template <int kUnitCost>
struct PackedWalk {
    uint32_t base;   // shared address: [S + 1] units (or positions) before each sequence, then [S] lengths
    int s, pos, end, count;

    __device__ static int at(uint32_t a) {
        int v;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
        return v;
    }

    __device__ void init(uint32_t base_, const PackedAttnParams &p) {
        base = base_;
        s = count = 0;
        const int total = at(base + 4 * p.num_seqs);
        if (p.balanced) {
            const int n = packed_sharers(total, gridDim.x), c = blockIdx.x;
            pos = c < n ? packed_share(total, c, n) : total;
            end = c < n ? packed_share(total, c + 1, n) : total;
        } else {
            pos = blockIdx.x;
            end = total;
        }
    }

    __device__ bool next(PackedUnit &x, const PackedAttnParams &p) {
        if (pos >= end) return false;
        const int lane = threadIdx.x & 31, S = p.num_seqs, groups = p.n_kv_heads >> p.log2_hpu;
        for (;;) {   // the sequence that holds pos, 32 candidates at a time
            const int c = s + 1 + lane;
            const unsigned m = __ballot_sync(kPackedAll, c > S || at(base + 4 * c) > pos);
            if (m) {
                s += __ffs(m) - 1;
                break;
            }
            s += 32;
        }
        x.s = s;
        const int L = at(base + 4 * (S + 1 + s));
        const int r = pos - at(base + 4 * s);
        if (p.balanced) {
            const int nt = (L + kPackedTile - 1) / kPackedTile, w = kUnitCost + nt;
            x.hg = r / w;
            const int from = r - x.hg * w, n = min(w - from, end - pos);
            const int a = max(from - kUnitCost, 0), b = from + n - kUnitCost;
            if (b <= a) return false;    // the share ends before the pair's first tile
            x.t0 = a * kPackedTile;
            x.t1 = min(L, b * kPackedTile);
            x.part = count == 0 ? 0 : 1;
            x.partial = !(a == 0 && b == nt);
            x.last = a == 0 ? pos - from + w - 1 : -1;
            pos += n;
        } else {
            x.part = r / groups;
            x.hg = r - x.part * groups;
            x.t0 = x.part * p.part_tokens;
            x.t1 = min(L, x.t0 + p.part_tokens);
            x.partial = L > p.part_tokens;
            x.last = -1;
            pos += gridDim.x;
        }
        ++count;
        return true;
    }
};

__device__ __forceinline__ uint4 packed_lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 packed_lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t packed_lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}

// Two fp32 lanes of work in one instruction: (a0, a1) = (x0, x1) * s + (a0, a1), and (x0, x1) * s.
__device__ __forceinline__ void fma2_by(float &a0, float &a1, float x0, float x1, float s) {
    asm("{\n\t.reg .b64 a, x, s;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\t"
        "fma.rn.f32x2 a, x, s, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1) : "f"(x0), "f"(x1), "f"(s));
}
__device__ __forceinline__ float2 mul2_by(float x0, float x1, float s) {
    float2 d;
    asm("{\n\t.reg .b64 x, s;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\t"
        "mul.rn.f32x2 x, x, s;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(x0), "f"(x1), "f"(s));
    return d;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) { return Elem<__half>::pack2(lo, hi); }

__device__ __forceinline__ float packed_max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <typename T>
__device__ __forceinline__ void store_quad(T *dst, float4 v, float inv) {
    *reinterpret_cast<uint2 *>(dst) =
        make_uint2(Elem<T>::pack2(v.x * inv, v.y * inv), Elem<T>::pack2(v.z * inv, v.w * inv));
}

// 1 / l for a row's sum; 0 for a row without keys (a NaN sum stays NaN).
__device__ __forceinline__ float packed_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

template <typename C>
__global__ void __launch_bounds__(kPackedThreads, C::kCtasPerSm) decode_packed_kernel(const __grid_constant__ PackedAttnParams p) {
    using T = typename C::Type;
    constexpr int D = C::kDim, B = C::kBlock, kUnitCost = C::kUnitCost;
    using Walk = PackedWalk<kUnitCost>;
    extern __shared__ __align__(128) uint8_t sm[];
    const uint32_t base = smem_addr(sm);
    const int S = p.num_seqs, H = 1 << p.log2_hpu, NS = p.stages;
    const int TL = kPackedConsumers >> p.log2_hpu;          // warps per kv head
    const int head_bytes = C::kHead, run = H * head_bytes;
    const int half = run * (kPackedTile / B);               // K (or V) of a stage
    const PackedSmem lay{2 * half, NS, S, D, TL > 1 ? 1 : 0};
    const uint32_t full0 = base + lay.bars(), empty0 = full0 + 8 * NS;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + lay.flag());
    int *scan = reinterpret_cast<int *>(sm + lay.scan());
    int *seq_base = reinterpret_cast<int *>(sm + lay.base());
    int *seq_len = reinterpret_cast<int *>(sm + lay.len());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int k = 0; k < NS; ++k) {
            mbar_init(full0 + 8 * k, 1);
            mbar_init(empty0 + 8 * k, kPackedConsumers);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    // lengths, tables and pools as the kernels before this one left them
    grid_dependency_wait();
    // the merge may start its launch; without one the next kernel may not (these
    // outputs may be what it reads first)
    if (p.merged) grid_launch_dependents();
    // ---- per sequence: length, and units (or positions) before it
    {
        const int cap = p.max_blocks * B, groups = p.n_kv_heads >> p.log2_hpu;
        const int per = (S + kPackedThreads - 1) / kPackedThreads;
        const int s0 = min(int(threadIdx.x) * per, S), s1 = min(s0 + per, S);
        int sum = 0;
        for (int s = s0; s < s1; ++s) {
            const int L = __ldg(p.context_lens + s), Lc = min(max(L, 0), cap);
            if (L != Lc && blockIdx.x == 0) atomicOr(p.err, PAGEDKV_DEVERR_CONTEXT_LEN);
            seq_len[s] = Lc;
            const int n = p.balanced ? (Lc > 0 ? (Lc + kPackedTile - 1) / kPackedTile + kUnitCost : 0)
                                     : (Lc > 0 ? (Lc + p.part_tokens - 1) / p.part_tokens : 1);
            sum += n * groups;
            seq_base[s + 1] = sum;
        }
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(kPackedAll, incl, d);
            if (lane >= d) incl += y;
        }
        if (lane == 31) scan[warp] = incl;
        if (threadIdx.x == 0) seq_base[0] = 0;
        __syncthreads();
        int before = incl - sum;
        for (int w = 0; w < warp; ++w) before += scan[w];
        for (int s = s0; s < s1; ++s) seq_base[s + 1] += before;
        __syncthreads();
    }
    Walk walk;
    walk.init(base + lay.base(), p);
    if (p.balanced) {
        // empty sequences have no unit: their rows are zeros
        for (int s = blockIdx.x; s < S; s += gridDim.x) {
            if (seq_len[s] != 0) continue;
            if (p.cuts_by_pair)
                for (int x = threadIdx.x; x < p.n_kv_heads >> p.log2_hpu; x += kPackedThreads)
                    p.ws_cuts[s * (p.n_kv_heads >> p.log2_hpu) + x] = make_int4(-1, 0, 0, 0);
            uint32_t *dst = reinterpret_cast<uint32_t *>(p.out) + size_t(s) * p.n_q_heads * (D / 2);
            for (int x = threadIdx.x; x < p.n_q_heads * (D / 2); x += kPackedThreads) dst[x] = 0u;
        }
    }

    if (warp == 0) {
        // -------------------------------------------------------- producer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        PackedUnit u;
        const int blk = lane >> 1, operand = lane & 1;     // this lane's copy of a tile
        const uint8_t *pool = operand ? p.v_cache : p.k_cache;
        const int lanes = 2 * (kPackedTile / B);
        const uint64_t once = l2_policy_evict_first();
        int4 cut = make_int4(-1, 0, 0, 0);
        while (ok && walk.next(u, p)) {
            const int32_t *table = p.block_tables + size_t(u.s) * p.max_blocks;
            const int h0 = u.hg << p.log2_hpu;
            // block ids of the next 32 blocks, one per lane
            int win = u.t0 / B;
            const int nblk = (u.t1 + B - 1) / B;
            int ids = win + lane < nblk ? __ldg(table + win + lane) : 0;
            for (int tok = u.t0; tok < u.t1; tok += kPackedTile) {
                const int j0 = tok / B;
                if (j0 + kPackedTile / B > win + 32) {
                    win = j0;
                    ids = win + lane < nblk ? __ldg(table + win + lane) : 0;
                }
                int pb = __shfl_sync(kPackedAll, ids, (j0 - win + blk) & 31);
                const int present = (min(kPackedTile, u.t1 - tok) + B - 1) / B;
                if (lane == 0) {
                    ok = !*abort_flag && mbar_wait(empty0 + 8 * stage, phase ^ 1u, p.err);
                    if (ok) mbar_arrive_expect_tx(full0 + 8 * stage, uint32_t(2 * present * run));
                }
                ok = __shfl_sync(kPackedAll, ok ? 1 : 0, 0) != 0;
                if (!ok) break;
                if (lane < lanes && blk < present) {
                    if (pb < 0 || pb >= p.num_blocks) {
                        atomicOr(p.err, PAGEDKV_DEVERR_BLOCK_ID);
                        pb = 0;
                    }
                    bulk_load_hint(base + stage * 2 * half + operand * half + blk * run,
                                   pool + (size_t(pb) * p.n_kv_heads + h0) * head_bytes, uint32_t(run),
                                   full0 + 8 * stage, once);
                }
                if (++stage == NS) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (p.balanced && u.last >= 0) {
                // for the merge: the pair, its first and last share, and the slot of its first piece
                const int total = Walk::at(base + lay.base() + 4 * S), n = packed_sharers(total, gridDim.x);
                const int pair = u.s * (p.n_kv_heads >> p.log2_hpu) + u.hg;
                const int4 mine = make_int4(u.partial ? pair : -1, blockIdx.x,
                                            u.partial ? packed_share_of(total, u.last, n) : 0, u.part);
                if (p.cuts_by_pair) {
                    if (lane == 0) p.ws_cuts[pair] = mine;
                } else if (u.partial) {
                    cut = mine;
                }
            }
        }
        if (p.balanced && !p.cuts_by_pair && lane == 0) p.ws_cuts[blockIdx.x] = cut;
        if (lane == 0) {
            // stop everyone if a wait ran out; then wait (bounded) for this CTA's
            // copies in flight, which consumers that stopped do not: each stage's
            // last use (the phase before a stage's first counts as done)
            if (!ok) *abort_flag = 1;
            for (int k = 0; k < NS; ++k) {
                mbar_wait(full0 + 8 * stage, phase ^ 1u, p.err);
                if (++stage == NS) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        return;
    }

    // ------------------------------------------------------------ consumers
    const int cw = warp - 1, hh = cw & (H - 1), tw = cw >> p.log2_hpu, g = p.group;
    C st;
    st.init(lane, hh, run);
    int stage = 0;
    uint32_t phase = 0;
    const T *q = reinterpret_cast<const T *>(p.q);
    T *out = reinterpret_cast<T *>(p.out);
    PackedUnit u;
    while (walk.next(u, p)) {
        const int qh0 = ((u.hg << p.log2_hpu) + hh) * g;
        st.begin(q, size_t(u.s) * p.n_q_heads + qh0, g, p.scale_log2);
        int i = 0;
        for (int tok = u.t0; tok < u.t1; tok += kPackedTile, ++i) {
            int good = mbar_try_wait(full0 + 8 * stage, phase);
            if (!good) good = !*abort_flag && mbar_wait(full0 + 8 * stage, phase, p.err);
            if (!__all_sync(kPackedAll, good)) {
                *abort_flag = 1;
            } else if ((i & (TL - 1)) == tw) {
                const uint32_t k = base + stage * 2 * half;
                if (u.t1 - tok >= kPackedTile) st.template tile<false>(k, k + half, run, kPackedTile);
                else st.template tile<true>(k, k + half, run, u.t1 - tok);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * stage);
            if (++stage == NS) {
                stage = 0;
                phase ^= 1u;
            }
        }
        st.finish();
        // row of head j: workspace rows [seq][q head][partition], or [CTA][slot][head of unit][j]
        auto ws_row = [&](int h, int j) {
            return p.balanced ? ((size_t(blockIdx.x) * 2 + u.part) * H + h) * g + j
                              : (size_t(u.s) * p.n_q_heads + size_t((u.hg << p.log2_hpu) + h) * g + j) * p.max_parts + u.part;
        };
        if (TL == 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = 2 * st.c + h;
                if (j >= g) continue;
                if (u.partial) {
                    const size_t row = ws_row(hh, j);
                    st.put_state(p.ws_o + row * D, h);
                    if (st.grp == 0) {
                        p.ws_m[row] = st.ref[h] * kLn2;
                        p.ws_l[row] = st.l[h];
                    }
                } else {
                    st.put_out(out + (size_t(u.s) * p.n_q_heads + qh0 + j) * D, h, packed_inverse(st.l[h]));
                }
            }
        } else {
            // the warps of a kv head join their states
            const int rowf = lay.row();
            float *jo = reinterpret_cast<float *>(sm + lay.join());
            float *jm = jo + kPackedConsumers * 8 * rowf, *jl = jm + kPackedConsumers * 8;
            named_barrier(1, 32 * kPackedConsumers);      // the previous unit's readers are done
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = 2 * st.c + h;
                if (j >= g) continue;
                st.put_state(jo + (cw * 8 + j) * rowf, h);
                if (st.grp == 0) {
                    jm[cw * 8 + j] = st.ref[h];
                    jl[cw * 8 + j] = st.l[h];
                }
            }
            named_barrier(1, 32 * kPackedConsumers);
            for (int x = threadIdx.x - 32; x < H * g * (D / 4); x += 32 * kPackedConsumers) {
                const int h = x / (g * (D / 4)), rem = x - h * g * (D / 4), j = rem / (D / 4), d = 4 * (rem - j * (D / 4));
                float M = -INFINITY;
                for (int t = 0; t < TL; ++t) M = fmaxf(M, jm[(t * H + h) * 8 + j]);
                float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
                float den = 0.f;
                for (int t = 0; t < TL; ++t) {
                    const int w = (t * H + h) * 8 + j;
                    // no tile of the unit was this warp's (a warp whose scores were all
                    // NaN has no reference either, and its NaN sums have to go through)
                    if (t >= i) continue;
                    const float f = fast_exp2(jm[w] - M);
                    const float4 v = *reinterpret_cast<const float4 *>(jo + w * rowf + d);
                    num.x = fmaf(f, v.x, num.x);
                    num.y = fmaf(f, v.y, num.y);
                    num.z = fmaf(f, v.z, num.z);
                    num.w = fmaf(f, v.w, num.w);
                    den = fmaf(f, jl[w], den);
                }
                if (u.partial) {
                    const size_t row = ws_row(h, j);
                    *reinterpret_cast<float4 *>(p.ws_o + row * D + d) = num;
                    if (d == 0) {
                        p.ws_m[row] = M * kLn2;
                        p.ws_l[row] = den;
                    }
                } else {
                    store_quad(out + (size_t(u.s) * p.n_q_heads + size_t((u.hg << p.log2_hpu) + h) * g + j) * D + d, num,
                               packed_inverse(den));
                }
            }
        }
    }
}

// Balanced split: the pieces of each (sequence, head group) that spans shares,
// joined by the softmax identity. Block x takes pair x, or, where the pairs
// outnumber the decode's CTAs, the pair that CTA x starts and does not end, of
// which there is at most one (ws_cuts, written by the decode). A
// row is kWarps warps' work (the launcher takes eight where a pair can have many
// pieces): each joins every kWarps-th piece, all loads of kBatch pieces in one
// round trip, against a running maximum of its own, and the warps' sums meet in
// shared memory.
template <int kWarps> constexpr int merge_pieces_threads() { return kWarps > 4 ? 32 * kWarps : 128; }

template <typename T, int D, int kWarps, int kBatch>
__global__ void __launch_bounds__(merge_pieces_threads<kWarps>()) merge_pieces_kernel(const __grid_constant__ PackedAttnParams p) {
    constexpr int E = D / 32, kRows = merge_pieces_threads<kWarps>() / 32 / kWarps;
    grid_dependency_wait();
    const int H = 1 << p.log2_hpu, rows = H * p.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * kRows + warp / kWarps, first = warp % kWarps;
    __shared__ float joined[merge_pieces_threads<kWarps>() / 32][D + 2];
    const int4 cut = __ldcg(p.ws_cuts + blockIdx.x);
    const int groups = p.n_kv_heads >> p.log2_hpu;
    if (cut.x < 0) return;
    // no cut at all, where a CTA of the decode stopped before it wrote one (a test
    // of its own: in one with the other it costs the merge 1 us)
    const bool bad = cut.x >= groups * p.num_seqs || cut.y < 0 || cut.z < cut.y || cut.z >= p.decode_ctas ||
                     (cut.w & ~1) != 0;
    if (bad) return;
    const int s = cut.x / groups, hg = cut.x - s * groups;
    const int c0 = cut.y, np = cut.z - c0 + 1, slot0 = cut.w;
    if (kWarps == 1 && r >= rows) return;
    float acc[E] = {}, M = -INFINITY, den = 0.f;
    if (r < rows) {
        for (int b = first; b < np; b += kBatch * kWarps) {
            float x[kBatch][E], m[kBatch], l[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = b + k * kWarps;
                m[k] = -INFINITY;
                l[k] = 0.f;
                if (i >= np) continue;
                const size_t row = (size_t(c0 + i) * 2 + (i == 0 ? slot0 : 0)) * rows + r;
                m[k] = __ldcg(p.ws_m + row) * kLog2e;
                l[k] = __ldcg(p.ws_l + row);
                const float *src = p.ws_o + row * D + lane * E;
                if constexpr (E == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
                    x[k][0] = v.x; x[k][1] = v.y; x[k][2] = v.z; x[k][3] = v.w;
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
                    x[k][0] = v.x; x[k][1] = v.y;
                }
            }
            float top = M;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) top = fmaxf(top, m[k]);
            const float alpha = M == -INFINITY ? 0.f : fast_exp2(M - top);
            M = top;
            den *= alpha;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= alpha;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (b + k * kWarps >= np) continue;
                const float w = fast_exp2(m[k] - M);
                den = fmaf(w, l[k], den);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(w, x[k][e], acc[e]);
            }
        }
    }
    if constexpr (kWarps > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) joined[warp][lane * E + e] = acc[e];
        if (lane == 0) {
            joined[warp][D] = M;
            joined[warp][D + 1] = den;
        }
        __syncthreads();
        if (first != 0 || r >= rows) return;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, joined[warp + w][D]);
        den = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w >= np) continue;                  // this warp had no piece
            const float f = fast_exp2(joined[warp + w][D] - top);
            den = fmaf(f, joined[warp + w][D + 1], den);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(f, joined[warp + w][lane * E + e], acc[e]);
        }
    }
    T *dst = reinterpret_cast<T *>(p.out) + (size_t(s) * p.n_q_heads + hg * rows + r) * D + lane * E;
    const float inv = packed_inverse(den);
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t *>(dst + e) = Elem<T>::pack2(acc[e] * inv, acc[e + 1] * inv);
}

template <typename C>
cudaError_t launch_decode_packed(PackedAttnParams p, int sms, cudaStream_t st) {
    using T = typename C::Type;
    constexpr int D = C::kDim;
    auto kernel = decode_packed_kernel<C>;
    const int H = 1 << p.log2_hpu, stage = 2 * H * (kPackedTile / C::kBlock) * C::kHead;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // as many stages as the CTAs of an SM leave room for in its 228 KB
    constexpr int kCtas = C::kCtasPerSm;
    PackedSmem lay{stage, 2, p.num_seqs, D, H < 4 ? 1 : 0};
    while (lay.stages < 8) {
        PackedSmem more = lay;
        ++more.stages;
        if (more.total() > 222 * 1024 / kCtas) break;
        lay = more;
    }
    p.stages = lay.stages;
    static std::atomic<unsigned long long> opened[kLaunchCacheDevices];
    e = open_dynamic_smem(opened, dev, kernel, lay.total());
    if (e != cudaSuccess) return e;
    static std::atomic<long long> fits[kLaunchCacheDevices];
    int per_sm = 0;
    e = occupancy_per_sm(fits, dev, kernel, kPackedThreads, lay.total(), &per_sm);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    if (per_sm > kCtas) per_sm = kCtas;
    const long long cap = (long long)p.max_blocks * p.block_size;
    const long long groups = p.n_kv_heads >> p.log2_hpu;
    const long long most = p.balanced ? groups * p.num_seqs * ((cap + kPackedTile - 1) / kPackedTile + C::kUnitCost)
                                      : groups * p.num_seqs * ((cap + p.part_tokens - 1) / p.part_tokens);
    const long long want = (long long)per_sm * sms;
    const int grid = int(most < want ? most : want);
    // (the pieces take at most 3 of the workspace's 8 CTAs per SM; the cuts lie behind them)
    const long long pairs = groups * p.num_seqs;
    p.cuts_by_pair = pairs <= grid ? 1 : 0;
    p.decode_ctas = grid;
    if (p.balanced) p.ws_cuts = reinterpret_cast<int4 *>(p.ws_o + size_t(grid) * 2 * (H * p.group) * D);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kPackedThreads);
    cfg.dynamicSmemBytes = size_t(lay.total());
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess || !p.balanced) return e;
    // A pair has about grid / pairs pieces: eight warps a row from eight on, and
    // batches that take them in one round trip up to 128; fewer loads a batch cost
    // less where there are fewer pieces. (Against batches of eight everywhere: one
    // request of 16000 tokens 15.4 us, now 13.4, 16 of 8000 36.1 and 35.1, 512 of
    // 500 43.3 and 42.3; 8 of 4000 14.7 and 15.1.)
    const unsigned rows = unsigned(H * p.group), blocks = unsigned(p.cuts_by_pair ? pairs : grid);
    const long long pieces = grid / pairs;
    cfg.dynamicSmemBytes = 0;
    auto merge = [&](auto merge_kernel, unsigned warps_per_row, int threads) {
        const unsigned per_block = unsigned(threads) / 32 / warps_per_row;
        cfg.blockDim = dim3(unsigned(threads));
        cfg.gridDim = dim3(blocks, (rows + per_block - 1) / per_block);
        return cudaLaunchKernelEx(&cfg, merge_kernel, p);
    };
    if (pieces >= 64) return merge(merge_pieces_kernel<T, D, 8, 16>, 8, merge_pieces_threads<8>());
    if (pieces >= 32) return merge(merge_pieces_kernel<T, D, 8, 8>, 8, merge_pieces_threads<8>());
    if (pieces >= 8) return merge(merge_pieces_kernel<T, D, 8, 2>, 8, merge_pieces_threads<8>());
    return merge(merge_pieces_kernel<T, D, 1, 2>, 1, merge_pieces_threads<1>());
}

}  // namespace pkv
