// api_common.h -- what the C ABI's translation units share (defined in api.cu).
#pragma once

#include <stdint.h>

namespace pkv {

// Error-word address and SM count of the current device; a pagedkv_status.
int api_device_state(unsigned int **err, int *sms);

inline bool api_aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

}  // namespace pkv
