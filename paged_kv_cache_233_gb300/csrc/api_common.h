// api_common.h -- what the C ABI's translation units share (defined in api.cu).
#pragma once

#include <cuda.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

struct PrefillParams;

// Error-word address and SM count of the current device; a pagedkv_status.
int api_device_state(unsigned int **err, int *sms);

// TMA view of a prefill call's queries for the tcgen05 kernel; a pagedkv_status.
int api_encode_q_map(CUtensorMap *map, const void *q, int dtype, int head_dim, int n_q_heads, int num_tokens,
                     int group);

// The key split of a prefill call whose other parameters p holds: sets p's
// key_parts and workspace arrays (key_parts, workspace as
// paged_attention_prefill_split takes them). A pagedkv_status.
int api_plan_key_split(PrefillParams &p, int key_parts, void *workspace, size_t workspace_bytes, int head_dim,
                       int max_query_len, int sms);

// Whether block tables, lengths, token lists and rows to append may be what a
// kernel of this library just ahead on the stream writes: a call with such results
// (paged_kv_build_tables, paged_kv_fork, paged_kv_release, the gathers of the packed
// caches) has been made in this process (they note it here). The
// 16-bit kernels then read them after their dependency wait; before it
// otherwise (with small steps in a graph the wait comes to a quarter of the rate:
// 16 slots of the batching trace 3.6 TB/s against 5.0).
bool api_late_inputs();
void api_note_device_inputs();

inline bool api_aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

}  // namespace pkv
