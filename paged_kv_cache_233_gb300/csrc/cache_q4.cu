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
// One thread owns a group: 64 bytes in, 16 bytes of codes and one (s, m) word
// out, no exchange between threads.
#include <math.h>

#include "q4.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;

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
    const T st = Pack<T>::toward_zero(__fdiv_rn(hi - lo, 15.f));
    const float s = Elem<T>::to_float(st);
    const T mt = Elem<T>::from_float(__fadd_rn(__fadd_rn(0.5f * lo, 0.5f * hi), 0.5f * s));
    const float m = Elem<T>::to_float(mt);
    pair = Pack<T>::bits(st) | (Pack<T>::bits(mt) << 16);
    if (s >= 0x1p-60f && s <= 0x1p60f) {
        // The quotient d / s: with r the remainder of its first estimate
        // q = d * (1 / s), exact in one fused multiply-add, q + r * (1 / s)
        // is exact wherever d / s is (a tie among them) and within an ulp
        // elsewhere. Adding 2^23 + 2^22 + 8 rounds it to a whole number, ties
        // to even, whose value plus 8 stands in the sum's low bits.
        const float inv = __fdiv_rn(1.f, s);
        const float2 inv2 = make_float2(inv, inv), ns2 = make_float2(-s, -s), nm2 = make_float2(-m, -m);
        const float2 magic = make_float2(12582920.f, 12582920.f);
        constexpr int kBase = 0x4b400000;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t acc = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 d = add2(Elem<T>::unpack2(w[4 * i + j]), nm2);
                const float2 q = mul2(d, inv2);
                const float2 r = fma2(q, ns2, d);
                const float2 t = add2(fma2(r, inv2, q), magic);
                const int a = min(max(__float_as_int(t.x), kBase), kBase + 15) - kBase;
                const int b = min(max(__float_as_int(t.y), kBase), kBase + 15) - kBase;
                acc += uint32_t(a) << (8 * j);
                acc += uint32_t(b) << (8 * j + 4);
            }
            codes[i] = acc;
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

// Where thread x's group lies: false for padding and bad slots.
template <int D>
__device__ __forceinline__ bool locate(const RowParams &p, unsigned int x, size_t &codes, size_t &pair) {
    constexpr int G = D / kQ4Group;
    const unsigned int t = x / p.per_token;
    const unsigned int hg = x - t * p.per_token;
    const int h = int(hg / G), g = int(hg % G);
    const long long slot = __ldg(reinterpret_cast<const long long *>(p.slots) + t);
    if (slot < 0) return false;
    if (slot >= p.num_slots) {
        if (hg == 0) atomicOr(p.err, PAGEDKV_DEVERR_SLOT_RANGE);
        return false;
    }
    const int B = 1 << p.log2_block;
    const int off = int(slot & (B - 1));
    const size_t base = (size_t(slot >> p.log2_block) * p.n_kv_heads + h) * q4_head_bytes(B, D);
    codes = base + size_t(g * B + off) * 16;
    pair = base + q4_pairs_at(B, D) + size_t(off * G + g) * 4;
    return true;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const __grid_constant__ RowParams p) {
    // every input may come from the kernel before this one (its slots from
    // paged_kv_build_tables); only then may the kernel after this one start
    grid_dependency_wait();
    grid_launch_dependents();
    const unsigned int x = blockIdx.x * kThreads + threadIdx.x;
    if (x >= p.count) return;
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
    size_t codes_at, pair_at;
    if (!locate<D>(p, x, codes_at, pair_at)) return;
    uint32_t c[4], pair;
    quantise<T>(w, c, pair);
    *reinterpret_cast<uint4 *>(p.cache[o] + codes_at) = make_uint4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<uint32_t *>(p.cache[o] + pair_at) = pair;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) gather_q4_kernel(const __grid_constant__ RowParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const unsigned int x = blockIdx.x * kThreads + threadIdx.x;
    if (x >= p.count) return;
    const int o = blockIdx.y;
    size_t codes_at, pair_at;
    if (!locate<D>(p, x, codes_at, pair_at)) return;
    const uint4 c = *reinterpret_cast<const uint4 *>(p.cache[o] + codes_at);
    const float2 sm = q4_pair<T>(*reinterpret_cast<const uint32_t *>(p.cache[o] + pair_at));
    const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
    uint4 *dst = reinterpret_cast<uint4 *>(p.rows[o]) + size_t(x) * 4;
    const float2 s2 = make_float2(sm.x, sm.x), m2 = make_float2(sm.y, sm.y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // 2^23 + c as a float, then c - 8 exactly
            const float a = __uint_as_float(and_or(cw[i] >> (8 * j), 15u, 0x4b000000u)) - 8388616.f;
            const float b = __uint_as_float(and_or(cw[i] >> (8 * j + 4), 15u, 0x4b000000u)) - 8388616.f;
            const float2 y = fma2(make_float2(a, b), s2, m2);
            r[j] = Elem<T>::pack2(y.x, y.y);
        }
        dst[i] = make_uint4(r[0], r[1], r[2], r[3]);
    }
}

// All tokens in launches of at most 2^31 groups per operand.
template <typename Kernel>
cudaError_t launch_rows(Kernel kernel, RowParams p, int num_tokens, int head_dim, cudaStream_t st) {
    const long long row_bytes = (long long)p.n_kv_heads * head_dim * 2;
    const int most = int((1ll << 31) / p.per_token);
    for (int t0 = 0; t0 < num_tokens; t0 += most) {
        const int n = num_tokens - t0 < most ? num_tokens - t0 : most;
        p.count = unsigned(n) * p.per_token;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((p.count + kThreads - 1) / kThreads, 2);
        cfg.blockDim = dim3(kThreads);
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
        if (e != cudaSuccess) return e;
        p.slots += n;
        for (int o = 0; o < 2; ++o) p.rows[o] = static_cast<uint8_t *>(p.rows[o]) + n * row_bytes;
        if (n == num_tokens - t0) break;
    }
    return cudaSuccess;
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
                             int block_size, long long num_slots, int dtype, int, unsigned int *err,
                             cudaStream_t st) {
    const RowParams p = row_params(slots, k_cache, v_cache, const_cast<void *>(k), const_cast<void *>(v),
                                   n_kv_heads, head_dim, block_size, num_slots, err);
    if (dtype == PAGEDKV_BF16)
        return head_dim == 64 ? launch_rows(append_q4_kernel<__nv_bfloat16, 64>, p, num_tokens, 64, st)
                              : launch_rows(append_q4_kernel<__nv_bfloat16, 128>, p, num_tokens, 128, st);
    return head_dim == 64 ? launch_rows(append_q4_kernel<__half, 64>, p, num_tokens, 64, st)
                          : launch_rows(append_q4_kernel<__half, 128>, p, num_tokens, 128, st);
}

cudaError_t launch_gather_q4(const uint8_t *k_cache, const uint8_t *v_cache, const int64_t *slots,
                             void *k, void *v, int num_tokens, int n_kv_heads, int head_dim,
                             int block_size, long long num_slots, int dtype, int, unsigned int *err,
                             cudaStream_t st) {
    const RowParams p = row_params(slots, const_cast<uint8_t *>(k_cache), const_cast<uint8_t *>(v_cache), k, v,
                                   n_kv_heads, head_dim, block_size, num_slots, err);
    if (dtype == PAGEDKV_BF16)
        return head_dim == 64 ? launch_rows(gather_q4_kernel<__nv_bfloat16, 64>, p, num_tokens, 64, st)
                              : launch_rows(gather_q4_kernel<__nv_bfloat16, 128>, p, num_tokens, 128, st);
    return head_dim == 64 ? launch_rows(gather_q4_kernel<__half, 64>, p, num_tokens, 64, st)
                          : launch_rows(gather_q4_kernel<__half, 128>, p, num_tokens, 128, st);
}

}  // namespace pkv
