// decode_q4.cuh -- fused paged-attention decode over the 4-bit cache (q4.h).
//
// Arithmetic. With c a code minus 8, s and m its group's scale and middle, a
// key's score and the output split into sums over the codes and sums over the
// pairs, so that no channel is ever multiplied by a scale:
//     q . K_t   = sum_g s_tg (q_g . c_tg)  +  sum_g m_tg (sum of q_g)
//     O[ch]     = sum_t (p_t s_tg) c_t[ch] +  sum_t p_t m_tg
// Codes are small integers, exact in fp16, and both contractions run on
// m16n8k16 tensor-core MMAs with fp32 sums: keys (or channels) are the 16 rows
// and the up to 8 query heads of the kv head the 8 columns. One 32-bit word
// from shared memory is 8 codes and one MMA operand pair; two and-or's, a
// shift and four fp16 adds or multiply-adds turn it into four operand
// registers. (Scaling each channel would cost as many instructions again, and
// a warp's instructions, not memory, are what bounds this kernel.)
//   K   an 8x8 matrix load gives lane (r, c) word c of token r's group: its
//       eight channels 8c .. 8c + 7. The MMA's k order is free as long as both
//       operands agree, so q is laid out once per unit to match. A group's two
//       MMAs accumulate q_g . (64 + code), which takes no arithmetic to make
//       from a code, one packed multiply-add per row applies s_tg, and one more
//       MMA adds sum_g m_tg Q_g - 72 s_tg Q_g with Q_g the sum of q_g: its rows
//       are the stored (s, m) pairs as they are, its columns Q_g and -72 Q_g in
//       two 16-bit parts. (An offset of 64 costs the fp32 sums 4 of their bits;
//       1024, which would save three more shifts, cost scores too many.)
//   V   the transposed 8x8 load gives lane (r, c) four channels 4r .. 4r + 3 of
//       tokens 2c and 2c + 1: two MMAs' rows. Probabilities are multiplied by
//       s_tg in fp32 and rounded once, to fp16, as the other operand. The m
//       part is summed in fp32; in bf16 caches with four groups, whose output
//       is rounded far more coarsely, it takes one more MMA instead: the
//       probabilities rounded to bf16, the pairs as stored.
// q is scaled by a power of two per row and taken as fp16, which holds every
// 8- or 11-bit significand: the MMAs are fp16 ones in bf16 caches too.
//
// Softmax reference. p = 2^(z - ref), and ref moves only when it must: when a
// p or a scale passes the bounds set with ref, whose product is 2^14 (fp16
// ends at 2^16). Then, with 2^e above the tile's largest scale, the bounds
// become 2^(12 - e) for p and 2^(e + 2) for scales, ref becomes the largest
// z_t + e_t - 4 of the tile's tokens, 2^e_t above token t's largest scale, if that
// is more, so that the largest p * s sits in the upper part of fp16's range
// whatever V's size, and the sums are rescaled. (With the largest z and the
// largest e of the tile, which can be two tokens', one token of little weight
// whose values were 10^6 times the others' took the others' products below
// fp16's range: 2% off, 10^8 times 24%.)
// Everything is relative to ref, so no result depends on when it moved beyond
// rounding.
//
// Work. A unit is (sequence, group of H kv heads, range of keys), split whole,
// in fixed partitions or in equal shares of the call's work per CTA: its 32-key
// tiles, and two tiles' worth (kQ4UnitCost) for each (sequence, head group),
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
// Measured (GB300, tables and lengths of a serving step; of a copy's 6.71 TB/s),
// and the copies alone, without arithmetic:
//   8 requests of 32768 to 131072 tokens, 8 kv heads of 128, 64 query heads,
//   fp16: 839 MB in 147.4 us, 5.69 TB/s (85%); copies 128.3 us
//   256 requests of 200 to 4000, 8 kv heads of 128, 32 query heads, bf16:
//   692 MB in 122.0 us, 5.68 TB/s (85%); copies 107.7
//   64 requests of 1 to 2048, 32 heads of 64, fp16, blocks of 8: 168 MB in
//   42.9 us, 3.93 TB/s (59%); copies 31.1
//   one request of 1999, 8 kv heads of 128: 8.5 us; copies 7.5
// The copies with their ramp, pieces and merge are most of a call; the consumers'
// instructions are what it takes beside them.
#pragma once

#include "decode_params.h"
#include "launch_cache.h"
#include "q4.cuh"

namespace pkv {

constexpr int kQ4Tile = 32;            // keys per stage
constexpr int kQ4Consumers = 4;
constexpr int kQ4Threads = 32 * (1 + kQ4Consumers);
constexpr int kQ4CtasPerSm = 3;
constexpr unsigned kQ4All = 0xffffffffu;

// Balanced split: the CTAs that get a share of `total` positions (tiles and unit
// costs), none of them empty, and share c's first position.
__device__ __forceinline__ int q4_sharers(int total, int grid) { return max(1, min(grid, total)); }
__device__ __forceinline__ int q4_share(int total, int c, int sharers) {
    return int((long long)total * c / sharers);
}

// The share that holds position t.
__device__ __forceinline__ int q4_share_of(int total, int t, int sharers) {
    int c = int((long long)t * sharers / total);
    while (c + 1 < sharers && q4_share(total, c + 1, sharers) <= t) ++c;
    while (c > 0 && q4_share(total, c, sharers) > t) --c;
    return c;
}

struct Q4Smem {
    int stage_bytes, stages, seqs, head_dim, shared_heads;   // shared_heads: warps of one kv head join states
    __host__ __device__ int bars() const { return stages * stage_bytes; }
    __host__ __device__ int flag() const { return bars() + 16 * stages; }
    __host__ __device__ int scan() const { return flag() + 16; }                 // a word per warp
    __host__ __device__ int base() const { return scan() + 32; }                 // seqs + 1
    __host__ __device__ int len() const { return base() + 4 * (seqs + 1); }      // seqs
    __host__ __device__ int join() const { return (len() + 4 * seqs + 15) & ~15; }
    __host__ __device__ int row() const { return head_dim + 4; }                 // floats of a joined row
    __host__ __device__ int total() const {
        return join() + (shared_heads ? kQ4Consumers * 8 * (row() + 2) * 4 : 0);
    }
};

struct Q4Unit {
    int s, hg, t0, t1;
    int part;         // its partition; balanced split: its piece slot of the CTA
    bool partial;     // the result is a state for the merge
    int last;         // balanced split: the position of the pair's last tile where this CTA has its first, else -1
};

// This CTA's units in order; the producer and every consumer warp walk a copy.
struct Q4Walk {
    uint32_t base;   // shared address: [S + 1] units (or positions) before each sequence, then [S] lengths
    int s, pos, end, count;

    __device__ static int at(uint32_t a) {
        int v;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
        return v;
    }

    __device__ void init(uint32_t base_, const Q4AttnParams &p) {
        base = base_;
        s = count = 0;
        const int total = at(base + 4 * p.num_seqs);
        if (p.balanced) {
            const int n = q4_sharers(total, gridDim.x), c = blockIdx.x;
            pos = c < n ? q4_share(total, c, n) : total;
            end = c < n ? q4_share(total, c + 1, n) : total;
        } else {
            pos = blockIdx.x;
            end = total;
        }
    }

    __device__ bool next(Q4Unit &x, const Q4AttnParams &p) {
        if (pos >= end) return false;
        const int lane = threadIdx.x & 31, S = p.num_seqs, groups = p.n_kv_heads >> p.log2_hpu;
        for (;;) {   // the sequence that holds pos, 32 candidates at a time
            const int c = s + 1 + lane;
            const unsigned m = __ballot_sync(kQ4All, c > S || at(base + 4 * c) > pos);
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
            const int nt = (L + kQ4Tile - 1) / kQ4Tile, w = kQ4UnitCost + nt;
            x.hg = r / w;
            const int from = r - x.hg * w, n = min(w - from, end - pos);
            const int a = max(from - kQ4UnitCost, 0), b = from + n - kQ4UnitCost;
            if (b <= a) return false;    // the share ends before the pair's first tile
            x.t0 = a * kQ4Tile;
            x.t1 = min(L, b * kQ4Tile);
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

__device__ __forceinline__ uint4 q4_lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 q4_lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t q4_lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}

// G (s, m) words of one token.
template <int G>
__device__ __forceinline__ void load_pairs(uint32_t a, uint32_t (&w)[G]) {
    if constexpr (G == 4) {
        const uint4 v = q4_lds128(a);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        const uint2 v = q4_lds64(a);
        w[0] = v.x; w[1] = v.y;
    }
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

// The scale (low half) of an (s, m) word, and the middle, as floats.
template <typename T>
__device__ __forceinline__ float scale_of(uint32_t w) {
    if constexpr (Elem<T>::kBf16) return __uint_as_float(w << 16);
    else return __half2float(__ushort_as_half(uint16_t(w)));
}
template <typename T>
__device__ __forceinline__ float middle_of(uint32_t w) {
    if constexpr (Elem<T>::kBf16) return __uint_as_float(w & 0xffff0000u);
    else return __half2float(__ushort_as_half(uint16_t(w >> 16)));
}

__device__ __forceinline__ float fmax3_q4(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// One consumer warp's state for a unit's kv head.
template <typename T, int D, int B>
struct Q4Consumer {
    static constexpr int G = D / kQ4Group;
    static constexpr int kPanel = B * 16;              // bytes between groups
    static constexpr int kPairs = B * D / 2;           // offset of the pairs in a (block, head)
    static constexpr int kHead = B * D * 5 / 8;

    uint32_t qb[G][4];     // q in the MMA's k order
    uint32_t qs0, qs1;     // the q sums' column words
    float kh[2];           // score scale of heads 2c, 2c + 1 (with the inverse of q's power of two)
    float o[G][2][4];
    // sum p m: this lane's part of it for each group, or (kMmaMiddle) the whole
    // sum of row grp of the pairs' halves (s0, m0, s1, ..) in [0][0], [0][1]
    static constexpr bool kMmaMiddle = Elem<T>::kBf16 && G == 4;
    float corr[kMmaMiddle ? 2 : G][2];
    float l[2];            // this lane's part of sum p
    float ref[2];
    float plim;            // the bounds: p, and scales as bits of T
    uint32_t slim;
    int grp, c;
    // this lane's offsets into a stage's K or V: its row of the matrix loads, of
    // the transposed ones, and the pairs of its rows, of its matrix row's word,
    // of token `lane`, and its row of the pairs' transposed loads
    uint32_t at_codes, at_trans, at_pairs, at_word, at_token, at_middle;

    __device__ void init(int lane, int hh, int run) {
        grp = lane >> 2;
        c = lane & 3;
        const int mi = lane >> 3, r8 = lane & 7;
        const uint32_t head = uint32_t(hh * kHead);
        at_codes = head + (G == 4 ? mi * kPanel : (mi & 1) * kPanel + octet(mi >> 1, run)) + r8 * 16;
        at_trans = head + octet(mi, run) + r8 * 16;
        at_pairs = head + kPairs + grp * 4 * G;
        at_word = at_pairs + (c & (G - 1)) * 4;
        at_middle = head + kPairs + octet_pairs(mi, run) + r8 * 4 * G;
        at_token = head + (lane / B) * run + kPairs + (lane % B) * 4 * G;
    }

    // Octet u of a tile (tokens 8u ..): its block's run and its row of codes, or pairs.
    __device__ static uint32_t octet(int u, int run) { return uint32_t((8 * u / B) * run + (8 * u % B) * 16); }
    __device__ static uint32_t octet_pairs(int u, int run) { return uint32_t((8 * u / B) * run + (8 * u % B) * 4 * G); }

    // Query rows qh0 .. qh0 + g - 1 of sequence s; column grp of the MMAs is head qh0 + grp.
    __device__ void begin(const T *q, size_t row0, int g, float scale_log2) {
        float x[G][8];
        float top = 0.f;
        const bool live = grp < g;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live) w = __ldg(reinterpret_cast<const uint4 *>(q + (row0 + grp) * D + 32 * i) + c);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = Elem<T>::unpack2(ww[j]);
                x[i][2 * j] = f.x;
                x[i][2 * j + 1] = f.y;
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        }
        top = fmaxf(top, __shfl_xor_sync(kQ4All, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kQ4All, top, 2));
        // a power of two that brings the row's largest value to [8, 16): 72
        // times a group's sum stays in fp16's range
        const int ex = min(max(int((__float_as_uint(top) >> 23) & 255u), 30), 240);
        const float mult = __uint_as_float(uint32_t(3 + 127 + 127 - ex) << 23);
        const float inv = __uint_as_float(uint32_t(ex - 3) << 23);   // 1 / mult
        float sums[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            sums[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                qb[i][j] = pack_f16(x[i][j] * mult, x[i][j + 4] * mult);
                const float2 f = Elem<__half>::unpack2(qb[i][j]);
                sums[i] += f.x + f.y;
            }
            sums[i] += __shfl_xor_sync(kQ4All, sums[i], 1);
            sums[i] += __shfl_xor_sync(kQ4All, sums[i], 2);
        }
        // the sums in two parts of the cache's type, under the pairs' halves;
        // the first MMA half takes lane c's group, and so does the second with
        // four groups, while with two groups lanes 2 and 3 hold the low parts
        float mine = sums[0];
#pragma unroll
        for (int i = 1; i < G; ++i)
            if ((c & (G - 1)) == i) mine = sums[i];
        const float off = -72.f * mine;
        const uint32_t whi = Elem<T>::pack2(off, mine);
        const float2 top2 = Elem<T>::unpack2(whi);
        const uint32_t wlo = Elem<T>::pack2(off - top2.x, mine - top2.y);
        qs0 = G == 4 || c < 2 ? whi : wlo;
        qs1 = G == 4 ? wlo : 0u;
        const float k = scale_log2 * inv;
        kh[0] = __shfl_sync(kQ4All, k, 8 * c);
        kh[1] = __shfl_sync(kQ4All, k, 8 * c + 4);
#pragma unroll
        for (auto &x : corr) x[0] = x[1] = 0.f;
#pragma unroll
        for (int i = 0; i < G; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][0][e] = o[i][1][e] = 0.f;
        }
        l[0] = l[1] = 0.f;
        ref[0] = ref[1] = -INFINITY;
        plim = -1.f;
        slim = 0;
    }

    // Move the reference and the bounds: sc the tile's sums of products, most the
    // bits of this lane's token's largest scale.
    __device__ __forceinline__ void move(const float (&sc)[4][2], uint32_t most, int nvalid) {
        // 2^e above the scale. It counts as at least the smallest that a bound can
        // hold, 2^-16 in fp16, whose bound 2^(e + 2) is then a normal number, and
        // 2^-32 in bf16: sums of p times middles of up to 2^64 then stay finite, and
        // products of p and scales of 2^-49 normal numbers. (NaN or infinite scales,
        // whose outputs are NaN, leave it at that.)
        constexpr float kLeast = Elem<T>::kBf16 ? 0x1p-32f : 0x1p-16f;
        const float s = scale_of<T>(most);
        const int mine = int(__float_as_uint(s < INFINITY ? fmaxf(s, kLeast) : kLeast) >> 23) - 126;
        const int e = __reduce_max_sync(kQ4All, mine);
        float top[2] = {-INFINITY, -INFINITY};   // the largest z_t + e_t - 4
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float up = float(__shfl_sync(kQ4All, mine, 8 * u + grp) - 4);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (8 * u + grp < nvalid) top[h] = fmaxf(top[h], fmaf(sc[u][h], kh[h], up));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int mask = 4; mask <= 16; mask <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(kQ4All, top[h], mask));
            const float nref = fmaxf(ref[h], top[h]);
            const float alpha = ref[h] == -INFINITY ? 0.f : fast_exp2(ref[h] - nref);
            ref[h] = nref;
            l[h] *= alpha;
#pragma unroll
            for (auto &x : corr) x[h] *= alpha;
#pragma unroll
            for (int i = 0; i < G; ++i) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    o[i][mt][h] *= alpha;
                    o[i][mt][2 + h] *= alpha;
                }
            }
        }
        plim = __uint_as_float(uint32_t(127 + 12 - e) << 23);
        const int f = e + 2;
        if constexpr (Elem<T>::kBf16) slim = f > 127 ? 0x7f7fu : uint32_t(f + 127) << 7;
        else slim = f > 15 ? 0x7bffu : uint32_t(f + 15) << 10;
    }

    // One tile: ks, vs the stage's K and V in shared memory, run the bytes between blocks.
    template <bool tail>
    __device__ __forceinline__ void tile(uint32_t ks, uint32_t vs, int run, int nvalid) {
        // ---- scores
        float sc[4][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            // words of octets 2t and 2t + 1, all groups
            uint32_t w[2][G];
            if constexpr (G == 4) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t r[4];
                    ldmatrix_x4(ks + at_codes + octet(2 * t + u, run), r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[u][i] = r[i];
                }
            } else {
                // (octets 2t and 2t + 1 lie as far apart as octets 0 and 1)
                uint32_t r[4];
                ldmatrix_x4(ks + at_codes + octet(2 * t, run), r);
                w[0][0] = r[0]; w[0][1] = r[1]; w[1][0] = r[2]; w[1][1] = r[3];
            }
            float s4[4];
            {
                // the m part: rows are the stored pairs
                uint32_t a[4];
                a[0] = q4_lds32(ks + at_word + octet_pairs(2 * t, run));
                a[1] = q4_lds32(ks + at_word + octet_pairs(2 * t + 1, run));
                a[2] = G == 4 ? a[0] : 0u;
                a[3] = G == 4 ? a[1] : 0u;
                mma_first<Elem<T>::kBf16>(s4, a, qs0, qs1);
            }
            uint32_t p0[G], p1[G];
            load_pairs<G>(ks + at_pairs + octet_pairs(2 * t, run), p0);
            load_pairs<G>(ks + at_pairs + octet_pairs(2 * t + 1, run), p1);
#pragma unroll
            for (int i = 0; i < G; ++i) {
                uint32_t x[4], y[4];
                q4_codes_64(w[0][i], x);
                q4_codes_64(w[1][i], y);
                float acc[4];
                const uint32_t a0[4] = {x[0], y[0], x[1], y[1]};
                const uint32_t a1[4] = {x[2], y[2], x[3], y[3]};
                mma_first<false>(acc, a0, qb[i][0], qb[i][1]);
                mma_m16n8k16<false>(acc, a1, qb[i][2], qb[i][3]);
                fma2_by(s4[0], s4[1], acc[0], acc[1], scale_of<T>(p0[i]));
                fma2_by(s4[2], s4[3], acc[2], acc[3], scale_of<T>(p1[i]));
            }
            sc[2 * t][0] = s4[0];
            sc[2 * t][1] = s4[1];
            sc[2 * t + 1][0] = s4[2];
            sc[2 * t + 1][1] = s4[3];
        }
        // ---- probabilities, and whether the reference has to move
        uint32_t most;   // the largest scale of token `lane`'s groups
        {
            uint32_t w[G];
            load_pairs<G>(vs + at_token, w);
            most = __vmaxu2(w[0], w[1]);
            if constexpr (G == 4) most = __vmaxu2(most, __vmaxu2(w[2], w[3]));
            most &= 0xffffu;
            if (tail && int(threadIdx.x & 31) >= nvalid) most = 0;
        }
        float pr[4][2];
        auto probabilities = [&]() {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float t = fmaf(sc[u][h], kh[h], -ref[h]);
                    if (tail && 8 * u + grp >= nvalid) t = -INFINITY;
                    pr[u][h] = fast_exp2(t);
                }
            }
        };
        probabilities();
        const float pm = fmax3_q4(fmax3_q4(pr[0][0], pr[0][1], pr[1][0]), fmax3_q4(pr[1][1], pr[2][0], pr[2][1]),
                                  fmaxf(pr[3][0], pr[3][1]));
        if (__any_sync(kQ4All, !(pm <= plim) || most > slim)) {
            move(sc, most, nvalid);
            probabilities();
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) fma2_by(l[0], l[1], pr[u][0], pr[u][1], 1.f);
        // ---- output
        if constexpr (kMmaMiddle) {
            // rows: the pairs' eight halves, two tokens a word (a row past them is not used)
            uint32_t r[4];
            ldmatrix_x4_trans(vs + at_middle, r);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if constexpr (tail) {
                    const int k0 = 16 * t + 2 * c;
                    r[2 * t] &= (k0 < nvalid ? 0xffffu : 0u) | (k0 + 1 < nvalid ? 0xffff0000u : 0u);
                    r[2 * t + 1] &= (k0 + 8 < nvalid ? 0xffffu : 0u) | (k0 + 9 < nvalid ? 0xffff0000u : 0u);
                }
                const uint32_t a[4] = {r[2 * t], 0u, r[2 * t + 1], 0u};
                float (&d)[4] = *reinterpret_cast<float(*)[4]>(&corr[0][0]);
                mma_m16n8k16<true>(d, a, movmatrix_trans(Elem<T>::pack2(pr[2 * t][0], pr[2 * t][1])),
                                   movmatrix_trans(Elem<T>::pack2(pr[2 * t + 1][0], pr[2 * t + 1][1])));
            }
        }
        uint32_t pw[4][G];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            load_pairs<G>(vs + at_pairs + octet_pairs(u, run), pw[u]);
            if (tail && 8 * u + grp >= nvalid) {
#pragma unroll
                for (int i = 0; i < G; ++i) pw[u][i] = 0;
            }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
            uint32_t b[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if constexpr (!kMmaMiddle)
                    fma2_by(corr[i][0], corr[i][1], pr[u][0], pr[u][1], middle_of<T>(pw[u][i]));
                const float2 v = mul2_by(pr[u][0], pr[u][1], scale_of<T>(pw[u][i]));
                b[u] = movmatrix_trans(pack_f16(v.x, v.y));
            }
            uint32_t r[4];
            ldmatrix_x4_trans(vs + at_trans + i * kPanel, r);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t x[4], y[4];
                q4_codes(r[2 * t], x);
                q4_codes(r[2 * t + 1], y);
                const uint32_t a0[4] = {x[0], x[1], y[0], y[1]};
                const uint32_t a1[4] = {x[2], x[3], y[2], y[3]};
                mma_m16n8k16<false>(o[i][0], a0, b[2 * t], b[2 * t + 1]);
                mma_m16n8k16<false>(o[i][1], a1, b[2 * t], b[2 * t + 1]);
            }
        }
    }

    // Sum the lanes' parts; afterwards o holds whole sums and l agrees in lanes of equal c.
    __device__ void finish() {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int mask = 4; mask <= 16; mask <<= 1) l[h] += __shfl_xor_sync(kQ4All, l[h], mask);
#pragma unroll
            for (int i = 0; i < G; ++i) {
                float x;
                if constexpr (kMmaMiddle) {
                    x = __shfl_sync(kQ4All, corr[0][h], 4 * (2 * i + 1) + c);   // row 2i + 1: group i's m
                } else {
                    x = corr[i][h];
#pragma unroll
                    for (int mask = 4; mask <= 16; mask <<= 1) x += __shfl_xor_sync(kQ4All, x, mask);
                }
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    o[i][mt][h] += x;
                    o[i][mt][2 + h] += x;
                }
            }
        }
    }

    // Four neighbouring channels of head 2c + h: 32 i + 4 grp ..
    __device__ float4 quad(int i, int h) const {
        return make_float4(o[i][0][h], o[i][0][2 + h], o[i][1][h], o[i][1][2 + h]);
    }
};

template <typename T>
__device__ __forceinline__ void store_quad(T *dst, float4 v, float inv) {
    *reinterpret_cast<uint2 *>(dst) =
        make_uint2(Elem<T>::pack2(v.x * inv, v.y * inv), Elem<T>::pack2(v.z * inv, v.w * inv));
}

// 1 / l for a row's sum; 0 for a row without keys (a NaN sum stays NaN).
__device__ __forceinline__ float q4_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

template <typename T, int D, int B>
__global__ void __launch_bounds__(kQ4Threads, kQ4CtasPerSm) decode_q4_kernel(const __grid_constant__ Q4AttnParams p) {
    constexpr int G = D / kQ4Group;
    extern __shared__ __align__(128) uint8_t sm[];
    const uint32_t base = smem_addr(sm);
    const int S = p.num_seqs, H = 1 << p.log2_hpu, NS = p.stages;
    const int TL = kQ4Consumers >> p.log2_hpu;          // warps per kv head
    const int head_bytes = q4_head_bytes(B, D), run = H * head_bytes;
    const int half = run * (kQ4Tile / B);               // K (or V) of a stage
    const Q4Smem lay{2 * half, NS, S, D, TL > 1 ? 1 : 0};
    const uint32_t full0 = base + lay.bars(), empty0 = full0 + 8 * NS;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + lay.flag());
    int *scan = reinterpret_cast<int *>(sm + lay.scan());
    int *seq_base = reinterpret_cast<int *>(sm + lay.base());
    int *seq_len = reinterpret_cast<int *>(sm + lay.len());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int k = 0; k < NS; ++k) {
            mbar_init(full0 + 8 * k, 1);
            mbar_init(empty0 + 8 * k, kQ4Consumers);
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
        const int per = (S + kQ4Threads - 1) / kQ4Threads;
        const int s0 = min(int(threadIdx.x) * per, S), s1 = min(s0 + per, S);
        int sum = 0;
        for (int s = s0; s < s1; ++s) {
            const int L = __ldg(p.context_lens + s), Lc = min(max(L, 0), cap);
            if (L != Lc && blockIdx.x == 0) atomicOr(p.err, PAGEDKV_DEVERR_CONTEXT_LEN);
            seq_len[s] = Lc;
            const int n = p.balanced ? (Lc > 0 ? (Lc + kQ4Tile - 1) / kQ4Tile + kQ4UnitCost : 0)
                                     : (Lc > 0 ? (Lc + p.part_tokens - 1) / p.part_tokens : 1);
            sum += n * groups;
            seq_base[s + 1] = sum;
        }
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(kQ4All, incl, d);
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
    Q4Walk walk;
    walk.init(base + lay.base(), p);
    if (p.balanced) {
        // empty sequences have no unit: their rows are zeros
        for (int s = blockIdx.x; s < S; s += gridDim.x) {
            if (seq_len[s] != 0) continue;
            if (p.cuts_by_pair)
                for (int x = threadIdx.x; x < p.n_kv_heads >> p.log2_hpu; x += kQ4Threads)
                    p.ws_cuts[s * (p.n_kv_heads >> p.log2_hpu) + x] = make_int4(-1, 0, 0, 0);
            uint32_t *dst = reinterpret_cast<uint32_t *>(p.out) + size_t(s) * p.n_q_heads * (D / 2);
            for (int x = threadIdx.x; x < p.n_q_heads * (D / 2); x += kQ4Threads) dst[x] = 0u;
        }
    }

    if (warp == 0) {
        // -------------------------------------------------------- producer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        Q4Unit u;
        const int blk = lane >> 1, operand = lane & 1;     // this lane's copy of a tile
        const uint8_t *pool = operand ? p.v_cache : p.k_cache;
        const int lanes = 2 * (kQ4Tile / B);
        const uint64_t once = l2_policy_evict_first();
        int4 cut = make_int4(-1, 0, 0, 0);
        while (ok && walk.next(u, p)) {
            const int32_t *table = p.block_tables + size_t(u.s) * p.max_blocks;
            const int h0 = u.hg << p.log2_hpu;
            // block ids of the next 32 blocks, one per lane
            int win = u.t0 / B;
            const int nblk = (u.t1 + B - 1) / B;
            int ids = win + lane < nblk ? __ldg(table + win + lane) : 0;
            for (int tok = u.t0; tok < u.t1; tok += kQ4Tile) {
                const int j0 = tok / B;
                if (j0 + kQ4Tile / B > win + 32) {
                    win = j0;
                    ids = win + lane < nblk ? __ldg(table + win + lane) : 0;
                }
                int pb = __shfl_sync(kQ4All, ids, (j0 - win + blk) & 31);
                const int present = (min(kQ4Tile, u.t1 - tok) + B - 1) / B;
                if (lane == 0) {
                    ok = !*abort_flag && mbar_wait(empty0 + 8 * stage, phase ^ 1u, p.err);
                    if (ok) mbar_arrive_expect_tx(full0 + 8 * stage, uint32_t(2 * present * run));
                }
                ok = __shfl_sync(kQ4All, ok ? 1 : 0, 0) != 0;
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
                const int total = Q4Walk::at(base + lay.base() + 4 * S), n = q4_sharers(total, gridDim.x);
                const int pair = u.s * (p.n_kv_heads >> p.log2_hpu) + u.hg;
                const int4 mine = make_int4(u.partial ? pair : -1, blockIdx.x,
                                            u.partial ? q4_share_of(total, u.last, n) : 0, u.part);
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
    Q4Consumer<T, D, B> st;
    st.init(lane, hh, run);
    int stage = 0;
    uint32_t phase = 0;
    const T *q = reinterpret_cast<const T *>(p.q);
    T *out = reinterpret_cast<T *>(p.out);
    Q4Unit u;
    while (walk.next(u, p)) {
        const int qh0 = ((u.hg << p.log2_hpu) + hh) * g;
        st.begin(q, size_t(u.s) * p.n_q_heads + qh0, g, p.scale_log2);
        int i = 0;
        for (int tok = u.t0; tok < u.t1; tok += kQ4Tile, ++i) {
            int good = mbar_try_wait(full0 + 8 * stage, phase);
            if (!good) good = !*abort_flag && mbar_wait(full0 + 8 * stage, phase, p.err);
            if (!__all_sync(kQ4All, good)) {
                *abort_flag = 1;
            } else if ((i & (TL - 1)) == tw) {
                const uint32_t k = base + stage * 2 * half;
                if (u.t1 - tok >= kQ4Tile) st.template tile<false>(k, k + half, run, kQ4Tile);
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
#pragma unroll
                    for (int i = 0; i < G; ++i)
                        *reinterpret_cast<float4 *>(p.ws_o + row * D + 32 * i + 4 * st.grp) = st.quad(i, h);
                    if (st.grp == 0) {
                        p.ws_m[row] = st.ref[h] * kLn2;
                        p.ws_l[row] = st.l[h];
                    }
                } else {
                    const float inv = q4_inverse(st.l[h]);
                    T *dst = out + (size_t(u.s) * p.n_q_heads + qh0 + j) * D + 4 * st.grp;
#pragma unroll
                    for (int i = 0; i < G; ++i) store_quad(dst + 32 * i, st.quad(i, h), inv);
                }
            }
        } else {
            // the warps of a kv head join their states
            const int rowf = lay.row();
            float *jo = reinterpret_cast<float *>(sm + lay.join());
            float *jm = jo + kQ4Consumers * 8 * rowf, *jl = jm + kQ4Consumers * 8;
            named_barrier(1, 32 * kQ4Consumers);      // the previous unit's readers are done
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = 2 * st.c + h;
                if (j >= g) continue;
#pragma unroll
                for (int i = 0; i < G; ++i)
                    *reinterpret_cast<float4 *>(jo + (cw * 8 + j) * rowf + 32 * i + 4 * st.grp) = st.quad(i, h);
                if (st.grp == 0) {
                    jm[cw * 8 + j] = st.ref[h];
                    jl[cw * 8 + j] = st.l[h];
                }
            }
            named_barrier(1, 32 * kQ4Consumers);
            for (int x = threadIdx.x - 32; x < H * g * (D / 4); x += 32 * kQ4Consumers) {
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
                               q4_inverse(den));
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
template <int kWarps> constexpr int q4_merge_threads() { return kWarps > 4 ? 32 * kWarps : 128; }

template <typename T, int D, int kWarps, int kBatch>
__global__ void __launch_bounds__(q4_merge_threads<kWarps>()) merge_q4_kernel(const __grid_constant__ Q4AttnParams p) {
    constexpr int E = D / 32, kRows = q4_merge_threads<kWarps>() / 32 / kWarps;
    grid_dependency_wait();
    const int H = 1 << p.log2_hpu, rows = H * p.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * kRows + warp / kWarps, first = warp % kWarps;
    __shared__ float joined[q4_merge_threads<kWarps>() / 32][D + 2];
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
    const float inv = q4_inverse(den);
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t *>(dst + e) = Elem<T>::pack2(acc[e] * inv, acc[e + 1] * inv);
}

template <typename T, int D, int B>
cudaError_t launch_decode_q4_sized(Q4AttnParams p, int sms, cudaStream_t st) {
    auto kernel = decode_q4_kernel<T, D, B>;
    const int H = 1 << p.log2_hpu, stage = 2 * H * kQ4Tile * D * 5 / 8;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // as many stages as the CTAs of an SM leave room for in its 228 KB
    constexpr int kCtas = kQ4CtasPerSm;
    Q4Smem lay{stage, 2, p.num_seqs, D, H < 4 ? 1 : 0};
    while (lay.stages < 8) {
        Q4Smem more = lay;
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
    e = occupancy_per_sm(fits, dev, kernel, kQ4Threads, lay.total(), &per_sm);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    if (per_sm > kCtas) per_sm = kCtas;
    const long long cap = (long long)p.max_blocks * p.block_size;
    const long long groups = p.n_kv_heads >> p.log2_hpu;
    const long long most = p.balanced ? groups * p.num_seqs * ((cap + kQ4Tile - 1) / kQ4Tile + kQ4UnitCost)
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
    cfg.blockDim = dim3(kQ4Threads);
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
    if (pieces >= 64) return merge(merge_q4_kernel<T, D, 8, 16>, 8, q4_merge_threads<8>());
    if (pieces >= 32) return merge(merge_q4_kernel<T, D, 8, 8>, 8, q4_merge_threads<8>());
    if (pieces >= 8) return merge(merge_q4_kernel<T, D, 8, 2>, 8, q4_merge_threads<8>());
    return merge(merge_q4_kernel<T, D, 1, 2>, 1, q4_merge_threads<1>());
}

template <typename T, int D>
cudaError_t launch_decode_q4_typed(const Q4AttnParams &p, int sms, cudaStream_t st) {
    return p.block_size == 8    ? launch_decode_q4_sized<T, D, 8>(p, sms, st)
           : p.block_size == 16 ? launch_decode_q4_sized<T, D, 16>(p, sms, st)
                                : launch_decode_q4_sized<T, D, 32>(p, sms, st);
}

}  // namespace pkv
