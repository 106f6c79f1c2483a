// decode_q8_f16.cu -- 8-bit decode with fp16 queries.
#include "decode_q8.cuh"

namespace pkv {

cudaError_t launch_decode_q8_f16(int head_dim, const PackedAttnParams &p, int sms, cudaStream_t st) {
    return head_dim == 64 ? launch_decode_q8_typed<__half, 64>(p, sms, st)
                          : launch_decode_q8_typed<__half, 128>(p, sms, st);
}

}  // namespace pkv
