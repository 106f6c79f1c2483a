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

#include "decode_packed.cuh"
#include "q4.cuh"

namespace pkv {

// G (s, m) words of one token.
template <int G>
__device__ __forceinline__ void load_pairs(uint32_t a, uint32_t (&w)[G]) {
    if constexpr (G == 4) {
        const uint4 v = packed_lds128(a);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        const uint2 v = packed_lds64(a);
        w[0] = v.x; w[1] = v.y;
    }
}

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

// One consumer warp's state for a unit's kv head.
template <typename T, int D, int B>
struct Q4Consumer {
    using Type = T;
    static constexpr int kDim = D, kBlock = B, kCtasPerSm = 3, kUnitCost = kQ4UnitCost;
    static constexpr int G = D / kQ4Group;
    static constexpr int kPanel = B * 16;              // bytes between groups
    static constexpr int kPairs = B * D / 2;           // offset of the pairs in a (block, head)
    static constexpr int kHead = q4_head_bytes(B, D);   // bytes of a (block, kv head)

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
        top = fmaxf(top, __shfl_xor_sync(kPackedAll, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kPackedAll, top, 2));
        // a power of two that brings the row's largest value to [8, 16): 72
        // times a group's sum stays in fp16's range
        const int ex = min(max(int((__float_as_uint(top) >> 23) & 255u), 30), 254);
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
            sums[i] += __shfl_xor_sync(kPackedAll, sums[i], 1);
            sums[i] += __shfl_xor_sync(kPackedAll, sums[i], 2);
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
        kh[0] = __shfl_sync(kPackedAll, k, 8 * c);
        kh[1] = __shfl_sync(kPackedAll, k, 8 * c + 4);
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
        const int e = __reduce_max_sync(kPackedAll, mine);
        float top[2] = {-INFINITY, -INFINITY};   // the largest z_t + e_t - 4
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float up = float(__shfl_sync(kPackedAll, mine, 8 * u + grp) - 4);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (8 * u + grp < nvalid) top[h] = fmaxf(top[h], fmaf(sc[u][h], kh[h], up));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int mask = 4; mask <= 16; mask <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(kPackedAll, top[h], mask));
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
                a[0] = packed_lds32(ks + at_word + octet_pairs(2 * t, run));
                a[1] = packed_lds32(ks + at_word + octet_pairs(2 * t + 1, run));
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
        const float pm = packed_max3(packed_max3(pr[0][0], pr[0][1], pr[1][0]), packed_max3(pr[1][1], pr[2][0], pr[2][1]),
                                  fmaxf(pr[3][0], pr[3][1]));
        if (__any_sync(kPackedAll, !(pm <= plim) || most > slim)) {
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
            for (int mask = 4; mask <= 16; mask <<= 1) l[h] += __shfl_xor_sync(kPackedAll, l[h], mask);
#pragma unroll
            for (int i = 0; i < G; ++i) {
                float x;
                if constexpr (kMmaMiddle) {
                    x = __shfl_sync(kPackedAll, corr[0][h], 4 * (2 * i + 1) + c);   // row 2i + 1: group i's m
                } else {
                    x = corr[i][h];
#pragma unroll
                    for (int mask = 4; mask <= 16; mask <<= 1) x += __shfl_xor_sync(kPackedAll, x, mask);
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
    // Head 2c + h's sums as a row of fp32, and times inv as a row of T.
    __device__ void put_state(float *row, int h) const {
#pragma unroll
        for (int i = 0; i < G; ++i) *reinterpret_cast<float4 *>(row + 32 * i + 4 * grp) = quad(i, h);
    }
    __device__ void put_out(T *row, int h, float inv) const {
#pragma unroll
        for (int i = 0; i < G; ++i) store_quad(row + 32 * i + 4 * grp, quad(i, h), inv);
    }
};


template <typename T, int D>
cudaError_t launch_decode_q4_typed(const PackedAttnParams &p, int sms, cudaStream_t st) {
    return p.block_size == 8    ? launch_decode_packed<Q4Consumer<T, D, 8>>(p, sms, st)
           : p.block_size == 16 ? launch_decode_packed<Q4Consumer<T, D, 16>>(p, sms, st)
                                : launch_decode_packed<Q4Consumer<T, D, 32>>(p, sms, st);
}

}  // namespace pkv
