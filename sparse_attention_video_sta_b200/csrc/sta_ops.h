// sta_ops.h -- what the plan-less operators (packed attention, 8-bit cache)
// share: argument checks, the per-device status word, and their launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sta.h"
#include "sta_internal.h"

namespace sta {

// Status of a CUDA error, its text kept for sta_last_error_detail (sta_api.cu).
sta_status op_cuda_status(cudaError_t e);
// Forget the calling thread's last CUDA error and make its device's context
// current (tensor maps are encoded through the driver API).
cudaError_t op_begin();
// Device address of the current device's status word (looked up once per device).
cudaError_t op_status_word(uint32_t** out);

// Time limit of every device-side wait of these operators' kernels, and whether a wait is made to
// run out (sta_debug_inject_operator_timeout).
struct OpWaits {
    uint64_t timeout_ns;
    int32_t inject;
};
OpWaits op_waits();

// A token-major bf16 tensor as the kernels address it.
struct Rows {
    __nv_bfloat16* p;
    int64_t ts, hs;  // elements from a token / a head to the next
};
inline Rows rows_of(const sta_rows* r) { return Rows{static_cast<__nv_bfloat16*>(r->data), r->token_stride, r->head_stride}; }

// Data pointer present and 16-byte aligned, strides positive multiples of 8
// elements (16 bytes: vector accesses and TMA strides).  A tensor without
// tokens is not read: it may have a null pointer.
inline bool rows_ok(const sta_rows* r, int64_t tokens) {
    if (r != nullptr && tokens == 0) return true;
    return r != nullptr && r->data != nullptr && reinterpret_cast<uintptr_t>(r->data) % 16 == 0 && r->token_stride > 0 &&
           r->head_stride > 0 && r->token_stride % 8 == 0 && r->head_stride % 8 == 0;
}

// Packed problem as the kernels take it.
struct PackedProblem {
    int32_t batch, heads, kv_heads, group;
    int32_t tokens_q, tokens_k;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int32_t causal, clear_tail;
    float scale;
    uint32_t* status;
    OpWaits waits;
};

// Checks shared by the packed calls; fills everything but `status`.
sta_status packed_problem(const sta_packed* p, bool pointers, PackedProblem* out);

// Pointers, alignment and counts of a cache (INVALID_ARG); sizes that this build has (UNSUPPORTED).
bool cache_ok(const sta_cache* c);
bool cache_supported(const sta_cache* c);

cudaError_t launch_packed_forward(const PackedProblem& p, int head_dim, const Rows& q, const Rows& k, const Rows& v,
                                  const Rows& o, float* lse, void* workspace, cudaStream_t stream);
cudaError_t launch_packed_backward(const PackedProblem& p, int head_dim, const Rows& q, const Rows& k, const Rows& v,
                                   const Rows& o, const Rows& dout, const float* lse, const Rows& dq, const Rows& dk,
                                   const Rows& dv, void* workspace, cudaStream_t stream);

}  // namespace sta
