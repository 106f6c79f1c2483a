// decode_q8.cuh -- the consumer of a decode over the 8-bit cache (q8.h,
// decode_packed.cuh).
//
// Arithmetic. A code is exact in fp16, and both contractions run on m16n8k16
// tensor-core MMAs with fp32 sums over the codes as they are: keys (or channels)
// are the 16 rows, the up to 8 query heads of the kv head the 8 columns. A block's
// scales 2^a (K) and 2^b (V) never touch a channel. A key's score is
//     z_t = (scale 2^a) (q . c_t),
// one factor per block and head, and the probabilities carry V's scale in their
// exponent:
//     w_t = 2^(z_t + b_t - ref),   O[ch] = sum_t w_t c_t[ch],   l = sum_t w_t 2^-b_t,
// the output O / l. Both scales being powers of two, no step of it rounds.
//   K   an 8x8 matrix load gives lane (r, c) the channels 4c .. 4c + 3 of token
//       r's panel: two conversions make them the two halves of an MMA's row. The
//       MMA's k order is free as long as both operands agree, so q is laid out
//       once per unit to match.
//   V   the transposed 8x8 load gives lane (r, c) the channels 2r, 2r + 1 of
//       tokens 2c and 2c + 1: a byte permutation pairs the tokens and two
//       conversions make rows r and r + 8 of an MMA. The probabilities are
//       rounded once, to fp16, as the other operand.
// q is scaled by a power of two per row and taken as fp16, which holds every
// 8- or 11-bit significand.
//
// Softmax reference. ref moves only when a w passes 2^15 (fp16 ends at 2^16), to
// the tile's largest z + b less 10, so that the largest w sits in the upper part of
// fp16's range whatever V's size; a w below 2^-24 of the largest loses bits.
// Everything is relative to ref, so no result depends on when it moved beyond
// rounding.
//
// Measured (one GB300, us; share of the copy bandwidth that the codes, scales, q and
// out come to):
//     256 x 200-4000 tokens, 8 heads of 128, 32 query heads, bf16     168    97%
//     8 x 32768-131072 tokens, 8 heads of 128, 64 query heads, fp16   201    98%
//     64 x 1-2048 tokens, 32 heads of 64, fp16, blocks of 8            48    84%
//     1 x 1999 tokens, 8 heads of 128, 32 query heads, bf16           7.6     8%
// The first two are the copies' (28% of the issue slots are used); the third is launch,
// ramp, pieces and merge beside them (37%); the last: two dependent launches. Two CTAs to
// an SM: three, as the 4-bit cache has, gained nothing, nor did two heads to a unit.
#pragma once

#include "decode_packed.cuh"
#include "q8.cuh"

namespace pkv {

// One consumer warp's state for a unit's kv head.
template <typename T, int D, int B>
struct Q8Consumer {
    using Type = T;
    static constexpr int kDim = D, kBlock = B, kCtasPerSm = 2, kUnitCost = kQ8UnitCost;
    static constexpr int kHead = q8_head_bytes(B, D);    // bytes of a (block, kv head)
    static constexpr int P = D / kQ8Panel;
    static constexpr int kPanel = B * kQ8Panel;          // bytes between panels
    static constexpr int kBlocks = kPackedTile / B;      // blocks of a tile
    static constexpr float kMost = 0x1p15f, kBelow = 10.f;

    uint32_t qb[P][2];     // q in the MMA's k order
    float kh[2];           // score scale of heads 2c, 2c + 1 (with the inverse of q's power of two)
    float o[P][4];         // channels 2 grp (.., ..) and 2 grp + 1 of the panel, heads 2c and 2c + 1
    float l[2];            // this lane's part of sum w / 2^b
    float ref[2];
    int grp, c;
    // this lane's offsets into a stage's K or V: its row of the matrix loads, of
    // the transposed ones, and the head's first block's scale
    uint32_t at_codes, at_trans, at_scale;

    // Octet u of a tile (tokens 8u ..): its block's run and its row of codes.
    __device__ static uint32_t octet(int u, int run) { return uint32_t((8 * u / B) * run + (8 * u % B) * kQ8Panel); }

    __device__ void init(int lane, int hh, int run) {
        grp = lane >> 2;
        c = lane & 3;
        const int mi = lane >> 3, r8 = lane & 7;
        const uint32_t head = uint32_t(hh * kHead);
        at_codes = head + (mi >> 1) * kPanel + octet(mi & 1, run) + r8 * 16;
        at_trans = head + octet(mi, run) + r8 * 16;
        at_scale = head + q8_scale_at(B, D);
    }

    // Query rows row0 .. row0 + g - 1; column grp of the MMAs is the grp-th.
    __device__ void begin(const T *q, size_t row0, int g, float scale_log2) {
        float x[P][4];
        float top = 0.f;
        const bool live = grp < g;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            uint2 w = make_uint2(0, 0);
            if (live) w = __ldg(reinterpret_cast<const uint2 *>(q + (row0 + grp) * D + 16 * i) + c);
            const float2 a = Elem<T>::unpack2(w.x), b = Elem<T>::unpack2(w.y);
            x[i][0] = a.x; x[i][1] = a.y; x[i][2] = b.x; x[i][3] = b.y;
#pragma unroll
            for (int j = 0; j < 4; ++j) top = fmaxf(top, fabsf(x[i][j]));
        }
        top = fmaxf(top, __shfl_xor_sync(kPackedAll, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kPackedAll, top, 2));
        // a power of two that brings the row's largest value to [2^14, 2^15)
        const int ex = min(max(int(__float_as_uint(top) >> 23), 30), 254);
        const float mult = __uint_as_float(uint32_t(14 + 127 + 127 - ex) << 23);
        const float k = scale_log2 * __uint_as_float(uint32_t(ex - 14) << 23);   // with 1 / mult
#pragma unroll
        for (int i = 0; i < P; ++i) {
            qb[i][0] = pack_f16(x[i][0] * mult, x[i][1] * mult);
            qb[i][1] = pack_f16(x[i][2] * mult, x[i][3] * mult);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
        }
        kh[0] = __shfl_sync(kPackedAll, k, 8 * c);
        kh[1] = __shfl_sync(kPackedAll, k, 8 * c + 4);
        l[0] = l[1] = 0.f;
        ref[0] = ref[1] = -INFINITY;
    }

    // Move the reference: z the tile's scores with V's exponents.
    __device__ __forceinline__ void move(const float (&z)[4][2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float top = fmaxf(fmaxf(z[0][h], z[1][h]), fmaxf(z[2][h], z[3][h]));
#pragma unroll
            for (int mask = 4; mask <= 16; mask <<= 1) top = fmaxf(top, __shfl_xor_sync(kPackedAll, top, mask));
            const float nref = fmaxf(ref[h], top - kBelow);
            const float alpha = ref[h] == -INFINITY ? 0.f : fast_exp2(ref[h] - nref);
            ref[h] = nref;
            l[h] *= alpha;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                o[i][h] *= alpha;
                o[i][2 + h] *= alpha;
            }
        }
    }

    // One tile: ks, vs the stage's K and V in shared memory, run the bytes between blocks.
    template <bool tail>
    __device__ __forceinline__ void tile(uint32_t ks, uint32_t vs, int run, int nvalid) {
        // ---- scores
        float z[4][2];
        float back[kBlocks];    // 2^-b
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                // panels i and i + 1 of octets 2t and 2t + 1
                uint32_t r[4];
                ldmatrix_x4(ks + at_codes + i * kPanel + octet(2 * t, run), r);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t a[4];
                    q8_halves(r[2 * j], a[0], a[2]);
                    q8_halves(r[2 * j + 1], a[1], a[3]);
                    mma_m16n8k16<false>(acc, a, qb[i + j][0], qb[i + j][1]);
                }
            }
            z[2 * t][0] = acc[0];
            z[2 * t][1] = acc[1];
            z[2 * t + 1][0] = acc[2];
            z[2 * t + 1][1] = acc[3];
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            // (a block past the context may hold anything, its scale too)
            const bool there = !tail || b * B < nvalid;
            const float sk = __uint_as_float(packed_lds32(ks + at_scale + b * run));
            const uint32_t sv = there ? packed_lds32(vs + at_scale + b * run) : 0x3f800000u;
            const float up = float(int(sv >> 23) - 127);
            back[b] = __uint_as_float(0x7f000000u - sv);
#pragma unroll
            for (int u = b * B / 8; u < (b + 1) * B / 8; ++u) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    z[u][h] = fmaf(z[u][h], kh[h] * sk, up);
                    if (tail && 8 * u + grp >= nvalid) z[u][h] = -INFINITY;
                }
            }
        }
        // ---- probabilities, and whether the reference has to move
        float pr[4][2];
        auto probabilities = [&]() {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int h = 0; h < 2; ++h) pr[u][h] = fast_exp2(z[u][h] - ref[h]);
            }
        };
        probabilities();
        const float pm = packed_max3(packed_max3(pr[0][0], pr[0][1], pr[1][0]), packed_max3(pr[1][1], pr[2][0], pr[2][1]),
                                     fmaxf(pr[3][0], pr[3][1]));
        if (__any_sync(kPackedAll, !(pm <= kMost))) {
            move(z);
            probabilities();
        }
        uint32_t b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            fma2_by(l[0], l[1], pr[u][0], pr[u][1], back[8 * u / B]);
            b[u] = movmatrix_trans(pack_f16(pr[u][0], pr[u][1]));
        }
        // ---- output
#pragma unroll
        for (int i = 0; i < P; ++i) {
            uint32_t r[4];
            ldmatrix_x4_trans(vs + at_trans + i * kPanel, r);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t a[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t w = r[2 * t + j];
                    if constexpr (tail) {   // what lies past the context may be a NaN
                        const int k0 = 16 * t + 8 * j + 2 * c;
                        w &= (k0 < nvalid ? 0xffffu : 0u) | (k0 + 1 < nvalid ? 0xffff0000u : 0u);
                    }
                    q8_halves(__byte_perm(w, 0, 0x3120), a[2 * j], a[2 * j + 1]);
                }
                mma_m16n8k16<false>(o[i], a, b[2 * t], b[2 * t + 1]);
            }
        }
    }

    // Sum the lanes' parts: afterwards l agrees in lanes of equal c.
    __device__ void finish() {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int mask = 4; mask <= 16; mask <<= 1) l[h] += __shfl_xor_sync(kPackedAll, l[h], mask);
        }
    }

    // Head 2c + h's sums as a row of fp32, and times inv as a row of T.
    __device__ void put_state(float *row, int h) const {
#pragma unroll
        for (int i = 0; i < P; ++i)
            *reinterpret_cast<float2 *>(row + 16 * i + 2 * grp) = make_float2(o[i][h], o[i][2 + h]);
    }
    __device__ void put_out(T *row, int h, float inv) const {
#pragma unroll
        for (int i = 0; i < P; ++i)
            *reinterpret_cast<uint32_t *>(row + 16 * i + 2 * grp) = Elem<T>::pack2(o[i][h] * inv, o[i][2 + h] * inv);
    }
};

template <typename T, int D>
cudaError_t launch_decode_q8_typed(const PackedAttnParams &p, int sms, cudaStream_t st) {
    return p.block_size == 8    ? launch_decode_packed<Q8Consumer<T, D, 8>>(p, sms, st)
           : p.block_size == 16 ? launch_decode_packed<Q8Consumer<T, D, 16>>(p, sms, st)
                                : launch_decode_packed<Q8Consumer<T, D, 32>>(p, sms, st);
}

}  // namespace pkv
