// decode_q8_bf16.cu -- 8-bit decode with bf16 queries.
#include "decode_q8.cuh"

namespace pkv {

cudaError_t launch_decode_q8_bf16(int head_dim, const PackedAttnParams &p, int sms, cudaStream_t st) {
    return head_dim == 64 ? launch_decode_q8_typed<__nv_bfloat16, 64>(p, sms, st)
                          : launch_decode_q8_typed<__nv_bfloat16, 128>(p, sms, st);
}

}  // namespace pkv
