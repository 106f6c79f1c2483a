// decode_q4_f16.cu -- 4-bit decode with fp16 queries and scales.
#include "decode_q4.cuh"

namespace pkv {

cudaError_t launch_decode_q4_f16(int head_dim, const PackedAttnParams &p, int sms, cudaStream_t st) {
    return head_dim == 64 ? launch_decode_q4_typed<__half, 64>(p, sms, st)
                          : launch_decode_q4_typed<__half, 128>(p, sms, st);
}

}  // namespace pkv
