// api_internal.h -- helpers shared by the host translation units of the
// library (not part of the C ABI: hidden from the shared library's exports).
#pragma once

#include <cuda_runtime.h>

#include "kvevict_ops.h"

#define KVEVICT_INTERNAL __attribute__((visibility("hidden")))

extern "C" {

// The CUDA device that holds the handle's state buffer (found once, at
// kvevict_create).
KVEVICT_INTERNAL int kvevict_handle_device(kvevict_t h);

// Every check kvevict_prefill_scored makes before it looks at the workspace:
// policy and dtype, the layer and its state, the prompt length, the Q/K/V
// pointers and their alignment, the launch limits. KVEVICT_OK or the status
// that call would return.
KVEVICT_INTERNAL int kvevict_prefill_scored_check(kvevict_t h, int layer, const void *Q, const void *K,
                                                  const void *V, int prompt_len);

// The device address of the allocation-free prefill's fixed scratch array on
// `device`, looked up once per device and cached; the lookup makes `device`
// current for its duration and restores the caller's device.
KVEVICT_INTERNAL int kvevict_static_scratch_address(int device, void **out);

// Shared-prefix attention whose suffix part the caller computes: `s` as for
// kvevict_shared_prefix_attention with k_rows = 0. _bytes: the workspace;
// _part: where in it the caller's part goes, fp32 outputs [batch][n_q_heads][d]
// and log2 normalisers [batch][n_q_heads] (every check of the call is made
// here); _run: the prefix's part and the join, after the caller's part on the
// same stream.
KVEVICT_INTERNAL int kvevict_prefix_bytes(const kvevict_shared_prefix_args *s, size_t *bytes);
KVEVICT_INTERNAL int kvevict_prefix_part(const kvevict_shared_prefix_args *s, float **part_o, float **part_l);
KVEVICT_INTERNAL int kvevict_prefix_run(const kvevict_shared_prefix_args *s, void *cuda_stream);

}  // extern "C"

namespace kvevict {

// The word on the current device for the errors of operator calls that give none
// of their own (kvevict_operator_errors). Its address is looked up once; also
// during a capture, where the lookup may have to load the library's kernels first.
KVEVICT_INTERNAL cudaError_t operator_errors_address(uint32_t **out);

}  // namespace kvevict
