// decode_q4_bf16.cu -- 4-bit decode with bf16 queries and scales.
#include "decode_q4.cuh"

namespace pkv {

cudaError_t launch_decode_q4_bf16(int head_dim, const PackedAttnParams &p, int sms, cudaStream_t st) {
    return head_dim == 64 ? launch_decode_q4_typed<__nv_bfloat16, 64>(p, sms, st)
                          : launch_decode_q4_typed<__nv_bfloat16, 128>(p, sms, st);
}

}  // namespace pkv
