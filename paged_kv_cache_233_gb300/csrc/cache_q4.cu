// cache_q4.cu -- rows into the 4-bit cache and back out of it.
//
// append: per group of 32 channels x_i of one token and kv head (q4.h), with
// lo and hi the smallest and largest of them,
//     s = (hi - lo) / 15 rounded towards zero to the 16-bit type,
//     m = lo / 2 + hi / 2 + s / 2 rounded to nearest,
//     c_i = clamp(round((x_i - m) / s), -8, 7) + 8, ties to even,
// so that code 0 stands for about lo and code 15 for about hi. The scale is
// rounded towards zero so that no code stands for more than the type's largest
// value when the group holds it. A group without spread (s = 0) holds m in
// every channel (code 8); a NaN or an infinity in a group makes its s NaN or
// infinite, and the whole group reads back as NaN.
// gather: x_i = s * (c_i - 8) + m, one rounding to the 16-bit type.
//
// append: a lane owns a group, 64 bytes in, 16 bytes of codes and one (s, m)
// word out. (Measured against it on 16383 tokens of 32 heads of 64, random
// slots, 41 us: two lanes per group, which read whole sectors but compute the
// scale twice, 43; groups streamed through shared memory by bulk copies, 51.)
// gather: four lanes per group, a word of eight codes each, and four groups a
// lane with their loads in flight together; a lane writes 16 bytes per group.
// (A lane per group, which writes a quarter of a sector at a time: 46 us there;
// four lanes and one group each, bound by latency: above 60; this form: 33.)
#include <math.h>

#include "q4.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;
constexpr int kGatherLanes = 4;     // lanes per group
constexpr int kGatherItems = 4;     // groups per lane

constexpr int kGatherPerCta = kThreads / kGatherLanes * kGatherItems;

// Two fp32 lanes of work in one instruction (sm_100 family).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// 16-bit types: packed smallest and largest (a NaN wins), and the roundings.
template <typename T> struct Pack;
template <> struct Pack<__half> {
    using T2 = __half2;
    __device__ static __half toward_zero(float x) { return __float2half_rz(x); }
    __device__ static uint32_t bits(__half x) { return __half_as_ushort(x); }
};
template <> struct Pack<__nv_bfloat16> {
    using T2 = __nv_bfloat162;
    __device__ static __nv_bfloat16 toward_zero(float x) { return __float2bfloat16_rz(x); }
    __device__ static uint32_t bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
};

// The 32 values of a group (16 words of two) -> its codes and its (s, m) word.
template <typename T>
__device__ __forceinline__ void quantise(const uint32_t (&w)[16], uint32_t (&codes)[4], uint32_t &pair) {
    using T2 = typename Pack<T>::T2;
    auto as2 = [](uint32_t x) { return *reinterpret_cast<T2 *>(&x); };
    T2 mn = as2(w[0]), mx = mn;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
        mn = __hmin2_nan(mn, as2(w[i]));
        mx = __hmax2_nan(mx, as2(w[i]));
    }
    const float lo = Elem<T>::to_float(__hmin_nan(mn.x, mn.y));
    const float hi = Elem<T>::to_float(__hmax_nan(mx.x, mx.y));
    const float spread = hi - lo;
    constexpr float kFifteenth = 1.f / 15.f;
    const float q15 = spread * kFifteenth;
    float s32 = fmaf(fmaf(q15, -15.f, spread), kFifteenth, q15);
    if (!(spread >= 0x1p-100f && spread <= 0x1p100f)) s32 = __fdiv_rn(spread, 15.f);
    const T st = Pack<T>::toward_zero(s32);
    const float s = Elem<T>::to_float(st);
    const T mt = Elem<T>::from_float(__fadd_rn(__fadd_rn(0.5f * lo, 0.5f * hi), 0.5f * s));
    const float m = Elem<T>::to_float(mt);
    pair = Pack<T>::bits(st) | (Pack<T>::bits(mt) << 16);
    constexpr int kBase = 0x4b400000;   // 2^23 + 2^22 as bits
    const float2 magic = make_float2(12582920.f, 12582920.f);
    if (s >= 0x1p-60f && s <= 0x1p60f) {
        // The quotient d / s, by Markstein's correction: with r the remainder of a
        // first estimate q = d * (1 / s), exact in one fused multiply-add, q + r * (1 / s) is
        // exact wherever d / s is (a tie among them) and within an ulp
        // elsewhere. Adding 2^23 + 2^22 + 8 rounds it to a whole number, ties
        // to even, whose value plus 8 stands in the sum's low bits.
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
        const float2 inv2 = make_float2(inv, inv), ns2 = make_float2(-s, -s), nm2 = make_float2(-m, -m);
        auto rounded = [&](float2 x) {
            const float2 d = add2(x, nm2);
            const float2 q = mul2(d, inv2);
            return add2(fma2(fma2(q, ns2, d), inv2, q), magic);
        };
        // the ends' codes: where they lie in 0 .. 15, so does every code between
        const float2 e = rounded(make_float2(lo, hi));
        if (__float_as_int(e.x) >= kBase && __float_as_int(e.y) <= kBase + 15) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t acc = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 t = rounded(Elem<T>::unpack2(w[4 * i + j]));
                    acc += __float_as_uint(t.x) * (1u << (8 * j));
                    acc += __float_as_uint(t.y) * (1u << (8 * j + 4));
                }
                codes[i] = acc - uint32_t(kBase) * 0x11111111u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t acc = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 t = rounded(Elem<T>::unpack2(w[4 * i + j]));
                    acc += uint32_t(min(max(__float_as_int(t.x), kBase), kBase + 15) - kBase) << (8 * j);
                    acc += uint32_t(min(max(__float_as_int(t.y), kBase), kBase + 15) - kBase) << (8 * j + 4);
                }
                codes[i] = acc;
            }
        }
        return;
    }
    // No spread, a NaN or an infinity: code 8. Scales whose reciprocal could
    // leave fp32's normal range (bf16 only): a division for each channel.
    const bool usable = s > 0.f && s <= 3.4028235e38f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t acc = 0x88888888u;
        if (usable) {
            acc = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = Elem<T>::unpack2(w[4 * i + j]);
                const float a = rintf(__fdiv_rn(x.x - m, s)), b = rintf(__fdiv_rn(x.y - m, s));
                acc |= uint32_t(int(fminf(fmaxf(a, -8.f), 7.f)) + 8) << (8 * j);
                acc |= uint32_t(int(fminf(fmaxf(b, -8.f), 7.f)) + 8) << (8 * j + 4);
            }
        }
        codes[i] = acc;
    }
}

struct RowParams {
    const int64_t *slots;
    uint8_t *cache[2];            // K, V
    void *rows[2];                // k, v [num_tokens][n_kv_heads][head_dim]
    unsigned int *err;
    unsigned int count;           // groups of all tokens of one operand
    unsigned int per_token;       // n_kv_heads * head_dim / 32
    int n_kv_heads, log2_block;
    long long num_slots;
};

// Where group x lies in its cache, given its token's slot: -1 for padding and bad slots.
struct Place {
    long long codes, pair;
};
template <int D>
__device__ __forceinline__ Place locate(const RowParams &p, unsigned int hg, long long slot) {
    constexpr int G = D / kQ4Group;
    Place at{-1, -1};
    if (slot < 0) return at;
    if (slot >= p.num_slots) {
        if (hg == 0) atomicOr(p.err, PAGEDKV_DEVERR_SLOT_RANGE);
        return at;
    }
    const int h = int(hg / G), g = int(hg % G), B = 1 << p.log2_block;
    const int off = int(slot & (B - 1));
    const long long base = ((slot >> p.log2_block) * p.n_kv_heads + h) * q4_head_bytes(B, D);
    at.codes = base + (g * B + off) * 16;
    at.pair = base + q4_pairs_at(B, D) + (off * G + g) * 4;
    return at;
}

// The slots of a thread's groups x0, x0 + step, .. (-1 past the last group),
// and their places among their tokens' groups.
template <int kItems>
__device__ __forceinline__ void load_slots(const RowParams &p, unsigned int x0, unsigned int step,
                                           long long (&slot)[kItems], unsigned int (&hg)[kItems]) {
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const unsigned int x = x0 + u * step, t = x / p.per_token;
        hg[u] = x - t * p.per_token;
        slot[u] = x < p.count ? __ldg(reinterpret_cast<const long long *>(p.slots) + t) : -1;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const __grid_constant__ RowParams p) {
    // every input may come from the kernel before this one (its slots from
    // paged_kv_build_tables); only then may the kernel after this one start
    grid_dependency_wait();
    grid_launch_dependents();
    // four neighbouring tokens to a group: their codes are 64 neighbouring bytes
    // where their slots are neighbours, as a prompt's are
    const unsigned int i0 = blockIdx.x * kThreads + threadIdx.x, quad = i0 / (4 * p.per_token);
    const unsigned int in = i0 - quad * 4 * p.per_token, t = quad * 4 + (in & 3), hg = in >> 2;
    const unsigned int x = t * p.per_token + hg;
    if (t >= p.count / p.per_token) return;
    const int o = blockIdx.y;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.rows[o]) + size_t(x) * 4;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 v = __ldcs(src + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
    const Place at = locate<D>(p, hg, __ldg(reinterpret_cast<const long long *>(p.slots) + t));
    if (at.codes < 0) return;
    uint32_t c[4], pair;
    quantise<T>(w, c, pair);
    *reinterpret_cast<uint4 *>(p.cache[o] + at.codes) = make_uint4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<uint32_t *>(p.cache[o] + at.pair) = pair;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) gather_q4_kernel(const __grid_constant__ RowParams p) {
    // (no early start for the kernel after this one: its work, rows of these to
    // append or attend over, comes after this grid's end)
    grid_dependency_wait();
    constexpr unsigned int kStep = kThreads / kGatherLanes;
    const unsigned int x0 = blockIdx.x * (kStep * kGatherItems) + threadIdx.x / kGatherLanes;
    const int o = blockIdx.y, word = threadIdx.x & 3;
    long long slot[kGatherItems];
    unsigned int hg[kGatherItems];
    load_slots<kGatherItems>(p, x0, kStep, slot, hg);
    uint32_t w[kGatherItems], sm[kGatherItems];
    bool put[kGatherItems];
#pragma unroll
    for (int u = 0; u < kGatherItems; ++u) {
        const Place at = locate<D>(p, hg[u], slot[u]);
        put[u] = at.codes >= 0;
        w[u] = put[u] ? *(reinterpret_cast<const uint32_t *>(p.cache[o] + at.codes) + word) : 0u;
        sm[u] = put[u] ? *reinterpret_cast<const uint32_t *>(p.cache[o] + at.pair) : 0u;
    }
#pragma unroll
    for (int u = 0; u < kGatherItems; ++u) {
        if (!put[u]) continue;
        uint32_t r[4];
        q4_values<T>(w[u], __byte_perm(sm[u], 0, 0x1010), __byte_perm(sm[u], 0, 0x3232), r);
        __stcs(reinterpret_cast<uint4 *>(p.rows[o]) + size_t(x0 + u * kStep) * 4 + word, make_uint4(r[0], r[1], r[2], r[3]));
    }
}

// All tokens in launches of at most 2^31 groups per operand; `launch` gets the
// launch's configuration and parameters.
template <typename Launch>
cudaError_t launch_rows(RowParams p, int num_tokens, int head_dim, cudaStream_t st, Launch launch) {
    const long long row_bytes = (long long)p.n_kv_heads * head_dim * 2;
    const int most = int((1ll << 31) / p.per_token);
    for (int t0 = 0; t0 < num_tokens; t0 += most) {
        const int n = num_tokens - t0 < most ? num_tokens - t0 : most;
        p.count = unsigned(n) * p.per_token;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.blockDim = dim3(kThreads);
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = launch(cfg, p);
        if (e != cudaSuccess) return e;
        p.slots += n;
        for (int o = 0; o < 2; ++o) p.rows[o] = static_cast<uint8_t *>(p.rows[o]) + n * row_bytes;
        if (n == num_tokens - t0) break;
    }
    return cudaSuccess;
}

template <typename T, int D>
cudaError_t append_typed(const RowParams &p, int num_tokens, cudaStream_t st) {
    return launch_rows(p, num_tokens, D, st, [&](cudaLaunchConfig_t &cfg, const RowParams &q) {
        const unsigned int quads = (q.count / q.per_token + 3) / 4;
        cfg.gridDim = dim3((quads * 4 * q.per_token + kThreads - 1) / kThreads, 2);
        return cudaLaunchKernelEx(&cfg, append_q4_kernel<T, D>, q);
    });
}

template <typename T, int D>
cudaError_t gather_typed(const RowParams &p, int num_tokens, cudaStream_t st) {
    return launch_rows(p, num_tokens, D, st, [&](cudaLaunchConfig_t &cfg, const RowParams &q) {
        cfg.gridDim = dim3((q.count + unsigned(kGatherPerCta) - 1) / unsigned(kGatherPerCta), 2);
        return cudaLaunchKernelEx(&cfg, gather_q4_kernel<T, D>, q);
    });
}

RowParams row_params(const int64_t *slots, uint8_t *kc, uint8_t *vc, void *k, void *v, int heads,
                     int head_dim, int block_size, long long num_slots, unsigned int *err) {
    RowParams p{};
    p.slots = slots;
    p.cache[0] = kc;
    p.cache[1] = vc;
    p.rows[0] = k;
    p.rows[1] = v;
    p.err = err;
    p.per_token = unsigned(heads) * unsigned(head_dim / kQ4Group);
    p.n_kv_heads = heads;
    while ((1 << p.log2_block) < block_size) ++p.log2_block;
    p.num_slots = num_slots;
    return p;
}

}  // namespace

cudaError_t launch_append_q4(const void *k, const void *v, const int64_t *slots, uint8_t *k_cache,
                             uint8_t *v_cache, int num_tokens, int n_kv_heads, int head_dim,
                             int block_size, long long num_slots, int dtype,
                             unsigned int *err, cudaStream_t st) {
    const RowParams p = row_params(slots, k_cache, v_cache, const_cast<void *>(k), const_cast<void *>(v),
                                   n_kv_heads, head_dim, block_size, num_slots, err);
    if (dtype == PAGEDKV_BF16)
        return head_dim == 64 ? append_typed<__nv_bfloat16, 64>(p, num_tokens, st)
                              : append_typed<__nv_bfloat16, 128>(p, num_tokens, st);
    return head_dim == 64 ? append_typed<__half, 64>(p, num_tokens, st)
                          : append_typed<__half, 128>(p, num_tokens, st);
}

cudaError_t launch_gather_q4(const uint8_t *k_cache, const uint8_t *v_cache, const int64_t *slots,
                             void *k, void *v, int num_tokens, int n_kv_heads, int head_dim,
                             int block_size, long long num_slots, int dtype,
                             unsigned int *err, cudaStream_t st) {
    const RowParams p = row_params(slots, const_cast<uint8_t *>(k_cache), const_cast<uint8_t *>(v_cache), k, v,
                                   n_kv_heads, head_dim, block_size, num_slots, err);
    if (dtype == PAGEDKV_BF16)
        return head_dim == 64 ? gather_typed<__nv_bfloat16, 64>(p, num_tokens, st)
                              : gather_typed<__nv_bfloat16, 128>(p, num_tokens, st);
    return head_dim == 64 ? gather_typed<__half, 64>(p, num_tokens, st)
                          : gather_typed<__half, 128>(p, num_tokens, st);
}

}  // namespace pkv
