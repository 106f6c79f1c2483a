// api_q4.cu -- the C ABI of the 4-bit paged cache and of the tables a step
// builds on the GPU (declared in include/pagedkv.h): host-side checks and
// launches.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "../../include/pagedkv.h"
#include "api_common.h"
#include "decode_launch.h"
#include "prefill.h"
#include "q4.h"

namespace {

using pkv::api_aligned;
using pkv::api_device_state;

constexpr int kMaxSeqs = 4096;
constexpr int kMaxCount = (1 << 30) - 1;   // free blocks and tokens of a step

int done(cudaError_t e) { return e == cudaSuccess ? PAGEDKV_OK : PAGEDKV_ERR_CUDA; }

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// The checks that every call on 4-bit pools shares.
int check_pool(int num_blocks, int block_size, int n_kv_heads, int head_dim, int dtype) {
    if (num_blocks < 1 || block_size < 1 || n_kv_heads < 1 || head_dim < 1 ||
        (dtype != PAGEDKV_F32 && dtype != PAGEDKV_F16 && dtype != PAGEDKV_BF16))
        return PAGEDKV_ERR_INVALID_ARG;
    if (dtype == PAGEDKV_F32) return PAGEDKV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PAGEDKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PAGEDKV_ERR_UNSUPPORTED;
    if (n_kv_heads > 65535) return PAGEDKV_ERR_UNSUPPORTED;
    return PAGEDKV_OK;
}

bool finite(float x) { return x == x && x != INFINITY && x != -INFINITY; }

// Whether a prefill call of `items` items of up to `tiles` key tiles each is
// faster with its keys shared out over the SMs: whole items take
// ceil(items / SMs) rounds of `tiles`, shared keys their even share, the extra
// pieces and a merge, which come to about 10 tiles and 0.2 per item. Items of
// several sequences count as one round: their lengths differ, which the host
// does not see, and whole items taken longest first then fill the SMs.
// `tiles` is the tables' width, not the contexts': exact where they are as wide.
// Measured (us, whole / shared; 8 kv heads, 32 query heads, bf16, 152 SMs; tables
// as wide as the longest context; the rule takes the smaller one each time):
//                                            heads of 128     heads of 64
//   one sequence  rows 33, cached 1000          25 / 19          21 / 15
//                 33, 6001                     111 / 25          96 / 18
//                 1216, 8192 (152 items)       163 / 188        138 / 151
//                 1280, 8192 (160)             288 / 196        245 / 159
//                 2048, 2048 (256)             110 / 140         92 / 112
//                 2048, 16384                  585 / 524        503 / 432
//   4 of 64 rows  up to 500 cached              17 / 21          14 / 17
//                 up to 4000                    47 / 29          39 / 22
//   20 of 64 rows up to 1000 (160 items)        26 / 56          21 / 43
//                 up to 4000                    76 / 103         63 / 74
bool split_pays(long long items, long long tiles, int seqs, int sms) {
    const long long rounds = seqs > 1 ? 1 : (items + sms - 1) / sms;
    const double gain = double(rounds * tiles) - double(items * tiles) / sms;
    return gain > 10.0 + 0.2 * double(items);
}

template <typename Launch>
int move_rows(const void *k, const void *v, const int64_t *slot_mapping, const void *k_cache,
              const void *v_cache, int num_tokens, int num_blocks, int block_size, int n_kv_heads,
              int head_dim, int dtype, Launch launch) {
    if (num_tokens < 0) return PAGEDKV_ERR_INVALID_ARG;
    int st = check_pool(num_blocks, block_size, n_kv_heads, head_dim, dtype);
    if (st != PAGEDKV_OK) return st;
    if (num_tokens == 0) return PAGEDKV_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PAGEDKV_ERR_INVALID_ARG;
    if (!api_aligned(k, 16) || !api_aligned(v, 16) || !api_aligned(k_cache, 16) ||
        !api_aligned(v_cache, 16) || !api_aligned(slot_mapping, 8))
        return PAGEDKV_ERR_INVALID_ARG;
    unsigned int *err = nullptr;
    int sms = 0;
    st = api_device_state(&err, &sms);
    if (st != PAGEDKV_OK) return st;
    return done(launch((long long)num_blocks * block_size, err));
}

}  // namespace

extern "C" {

int paged_kv_build_tables(const int32_t *new_lens, const int32_t *context_lens, int32_t *block_tables,
                          const int32_t *free_blocks, const int32_t *free_count, int32_t *query_start,
                          int32_t *token_seq, int32_t *token_pos, int64_t *slot_mapping,
                          int32_t *context_lens_out, int32_t *free_count_out, int num_seqs,
                          int max_blocks_per_seq, int free_capacity, int token_capacity, int block_size,
                          int num_blocks, void *stream) {
    if (num_seqs < 0 || max_blocks_per_seq < 1 || free_capacity < 0 || token_capacity < 0 ||
        block_size < 1 || num_blocks < 1)
        return PAGEDKV_ERR_INVALID_ARG;
    if (num_seqs > kMaxSeqs || free_capacity > kMaxCount || token_capacity > kMaxCount ||
        (long long)max_blocks_per_seq * block_size > INT_MAX / 2)
        return PAGEDKV_ERR_UNSUPPORTED;
    if (!free_count || !query_start || !free_count_out) return PAGEDKV_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!new_lens || !context_lens || !block_tables || !context_lens_out))
        return PAGEDKV_ERR_INVALID_ARG;
    if ((free_capacity > 0 && !free_blocks) || (token_capacity > 0 && (!token_seq || !token_pos)))
        return PAGEDKV_ERR_INVALID_ARG;
    if (!api_aligned(new_lens, 4) || !api_aligned(context_lens, 4) || !api_aligned(block_tables, 4) ||
        !api_aligned(free_blocks, 4) || !api_aligned(free_count, 4) || !api_aligned(query_start, 4) ||
        !api_aligned(token_seq, 4) || !api_aligned(token_pos, 4) || !api_aligned(slot_mapping, 8) ||
        !api_aligned(context_lens_out, 4) || !api_aligned(free_count_out, 4))
        return PAGEDKV_ERR_INVALID_ARG;
    pkv::api_note_device_inputs();   // before the launch: calls that read these tables come later
    pkv::TablesParams p{};
    int sms = 0;
    const int st = api_device_state(&p.err, &sms);
    if (st != PAGEDKV_OK) return st;
    p.new_lens = new_lens;
    p.context_lens = context_lens;
    p.block_tables = block_tables;
    p.free_blocks = free_blocks;
    p.free_count = free_count;
    p.query_start = query_start;
    p.token_seq = token_seq;
    p.token_pos = token_pos;
    p.slot_mapping = slot_mapping;
    p.context_lens_out = context_lens_out;
    p.free_count_out = free_count_out;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.free_capacity = free_capacity;
    p.token_capacity = token_capacity;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    return done(pkv::launch_build_tables(p, sms, static_cast<cudaStream_t>(stream)));
}

int paged_kv_append_q4(const void *k, const void *v, const int64_t *slot_mapping, void *k_cache,
                       void *v_cache, int num_tokens, int num_blocks, int block_size, int n_kv_heads,
                       int head_dim, int dtype, void *stream) {
    return move_rows(k, v, slot_mapping, k_cache, v_cache, num_tokens, num_blocks, block_size, n_kv_heads,
                     head_dim, dtype, [&](long long num_slots, unsigned int *err) {
                         return pkv::launch_append_q4(k, v, slot_mapping, static_cast<uint8_t *>(k_cache),
                                                      static_cast<uint8_t *>(v_cache), num_tokens, n_kv_heads,
                                                      head_dim, block_size, num_slots, dtype, err,
                                                      static_cast<cudaStream_t>(stream));
                     });
}

int paged_kv_gather_q4(const void *k_cache, const void *v_cache, const int64_t *slot_mapping, void *k,
                       void *v, int num_tokens, int num_blocks, int block_size, int n_kv_heads,
                       int head_dim, int dtype, void *stream) {
    return move_rows(k, v, slot_mapping, k_cache, v_cache, num_tokens, num_blocks, block_size, n_kv_heads,
                     head_dim, dtype, [&](long long num_slots, unsigned int *err) {
                         pkv::api_note_device_inputs();   // as above: calls that append these rows
                         return pkv::launch_gather_q4(static_cast<const uint8_t *>(k_cache),
                                                      static_cast<const uint8_t *>(v_cache), slot_mapping, k, v,
                                                      num_tokens, n_kv_heads, head_dim, block_size, num_slots,
                                                      dtype, err, static_cast<cudaStream_t>(stream));
                     });
}

int paged_attention_decode_q4(const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *block_tables, const int32_t *context_lens, float scale,
                              void *out, int num_seqs, int n_q_heads, int n_kv_heads, int head_dim,
                              int num_blocks, int block_size, int max_blocks_per_seq, int partition_tokens,
                              void *workspace, size_t workspace_bytes, int dtype, void *stream) {
    if (num_seqs < 0 || n_q_heads < 1 || max_blocks_per_seq < 1 ||
        (partition_tokens < 0 && partition_tokens != PAGEDKV_PARTITION_BALANCED))
        return PAGEDKV_ERR_INVALID_ARG;
    int st = check_pool(num_blocks, block_size, n_kv_heads, head_dim, dtype);
    if (st == PAGEDKV_ERR_INVALID_ARG) return st;
    if (n_q_heads % n_kv_heads != 0 || !finite(scale)) return PAGEDKV_ERR_INVALID_ARG;
    if (partition_tokens > 0 && partition_tokens % 32 != 0) return PAGEDKV_ERR_INVALID_ARG;
    if (st != PAGEDKV_OK) return st;
    const int group = n_q_heads / n_kv_heads;
    const long long cap = (long long)max_blocks_per_seq * block_size;
    if (group > 8 || num_seqs > kMaxSeqs || cap > INT_MAX / 2) return PAGEDKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PAGEDKV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out) return PAGEDKV_ERR_INVALID_ARG;
    if (!api_aligned(q, 16) || !api_aligned(k_cache, 16) || !api_aligned(v_cache, 16) ||
        !api_aligned(out, 16) || !api_aligned(block_tables, 4) || !api_aligned(context_lens, 4))
        return PAGEDKV_ERR_INVALID_ARG;
    if (partition_tokens != 0) {
        const size_t need = paged_attention_workspace_bytes(num_seqs, n_q_heads, head_dim, max_blocks_per_seq,
                                                            block_size, partition_tokens);
        if (need == 0 || !workspace || workspace_bytes < need || !api_aligned(workspace, 256))
            return PAGEDKV_ERR_WORKSPACE;
    }
    pkv::Q4AttnParams p{};
    int sms = 0;
    st = api_device_state(&p.err, &sms);
    if (st != PAGEDKV_OK) return st;
    p.q = q;
    p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.v_cache = static_cast<const uint8_t *>(v_cache);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.out = out;
    p.scale_log2 = scale * pkv::kLog2e;
    p.num_seqs = num_seqs;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = group;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    while ((1 << p.log2_block) < block_size) ++p.log2_block;
    p.max_blocks = max_blocks_per_seq;
    p.balanced = partition_tokens == PAGEDKV_PARTITION_BALANCED ? 1 : 0;
    p.log2_hpu = n_kv_heads % 4 == 0 ? 2 : (n_kv_heads % 2 == 0 ? 1 : 0);
    // (unsplit: one partition of the tables' whole width)
    p.part_tokens = partition_tokens > 0 ? partition_tokens : int((cap + 31) / 32 * 32);
    p.max_parts = int((cap + p.part_tokens - 1) / p.part_tokens);
    p.merged = p.balanced || p.max_parts > 1 ? 1 : 0;
    // the kernel counts units and tiles in ints
    const long long units = (long long)num_seqs * (n_kv_heads >> p.log2_hpu) *
                            (p.balanced ? (cap + 31) / 32 + pkv::kQ4UnitCost : p.max_parts);
    if (units > INT_MAX / 2) return PAGEDKV_ERR_UNSUPPORTED;
    if (partition_tokens != 0) {
        // rows of partition states, or of pieces: two per CTA, as paged_attention_workspace_bytes sizes them
        const size_t rows = p.balanced ? size_t(16) * sms * size_t(n_q_heads < 32 ? n_q_heads : 32)
                                       : size_t(num_seqs) * n_q_heads * size_t(p.max_parts);
        uint8_t *w = static_cast<uint8_t *>(workspace);
        p.ws_o = reinterpret_cast<float *>(w);
        p.ws_m = reinterpret_cast<float *>(w + round256(rows * head_dim * 4));
        p.ws_l = reinterpret_cast<float *>(w + round256(rows * head_dim * 4) + round256(rows * 4));
    }
    cudaError_t e = dtype == PAGEDKV_BF16
                        ? pkv::launch_decode_q4_bf16(head_dim, p, sms, static_cast<cudaStream_t>(stream))
                        : pkv::launch_decode_q4_f16(head_dim, p, sms, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess && p.merged && !p.balanced)
        e = pkv::launch_lse_merge(dtype, head_dim, p.ws_o, p.ws_m, p.ws_l, context_lens, out, num_seqs, n_q_heads,
                                  p.part_tokens, p.max_parts, int(cap), p.err, static_cast<cudaStream_t>(stream));
    return done(e);
}

int paged_attention_prefill_q4(const void *q, const void *k_cache, const void *v_cache,
                               const int32_t *block_tables, const int32_t *query_start,
                               const int32_t *context_lens, float scale, void *out, int num_seqs,
                               int num_tokens, int max_query_len, int n_q_heads, int n_kv_heads, int head_dim,
                               int num_blocks, int block_size, int max_blocks_per_seq, int dtype,
                               int key_parts, void *workspace, size_t workspace_bytes, void *stream) {
    if (key_parts < 0 || key_parts > 32 || num_seqs < 0 || num_tokens < 0 || max_query_len < 0 ||
        n_q_heads < 1 || max_blocks_per_seq < 1)
        return PAGEDKV_ERR_INVALID_ARG;
    int st = check_pool(num_blocks, block_size, n_kv_heads, head_dim, dtype);
    if (st == PAGEDKV_ERR_INVALID_ARG) return st;
    if (n_q_heads % n_kv_heads != 0 || !finite(scale)) return PAGEDKV_ERR_INVALID_ARG;
    if (st != PAGEDKV_OK) return st;
    const int group = n_q_heads / n_kv_heads;
    const long long cap = (long long)max_blocks_per_seq * block_size;
    if (group > 64 || num_seqs > 65535 || cap > INT_MAX / 2) return PAGEDKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0 || max_query_len == 0) return PAGEDKV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !query_start || !context_lens || !out)
        return PAGEDKV_ERR_INVALID_ARG;
    if (!api_aligned(q, 16) || !api_aligned(k_cache, 16) || !api_aligned(v_cache, 16) ||
        !api_aligned(out, 16) || !api_aligned(block_tables, 4) || !api_aligned(query_start, 4) ||
        !api_aligned(context_lens, 4))
        return PAGEDKV_ERR_INVALID_ARG;
    pkv::PrefillParams p{};
    int sms = 0;
    st = api_device_state(&p.err, &sms);
    if (st != PAGEDKV_OK) return st;
    p.q = q;
    p.k_q4 = static_cast<const uint8_t *>(k_cache);
    p.v_q4 = static_cast<const uint8_t *>(v_cache);
    p.block_tables = block_tables;
    p.query_start = query_start;
    p.context_lens = context_lens;
    p.out = out;
    p.scale_log2 = scale * pkv::kLog2e;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = group;
    p.tile_tokens = 2 * (128 / group);
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    while ((1 << p.log2_block) < block_size) ++p.log2_block;
    p.max_blocks = max_blocks_per_seq;
    // the persistent kernel counts its work items in ints
    const long long per_seq = ((long long)max_query_len + p.tile_tokens - 1) / p.tile_tokens * n_kv_heads;
    if (per_seq > (INT_MAX / 2) / num_seqs) return PAGEDKV_ERR_UNSUPPORTED;
    if (key_parts == 0)
        key_parts = workspace && workspace_bytes >= paged_attention_prefill_workspace_bytes(head_dim) &&
                            split_pays(per_seq * num_seqs, (cap + 63) / 64, num_seqs, sms)
                        ? 32
                        : 1;
    st = pkv::api_plan_key_split(p, key_parts, workspace, workspace_bytes, head_dim, max_query_len, sms);
    if (st != PAGEDKV_OK) return st;
    CUtensorMap qmap;
    st = pkv::api_encode_q_map(&qmap, q, dtype, head_dim, n_q_heads, num_tokens, group);
    if (st != PAGEDKV_OK) return st;
    cudaError_t e = pkv::launch_prefill_q4_tc(dtype, head_dim, qmap, p, max_query_len, sms,
                                              static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess && p.key_parts > 1)
        e = pkv::launch_prefill_merge(dtype, head_dim, p, max_query_len, sms, static_cast<cudaStream_t>(stream));
    return done(e);
}

}  // extern "C"
