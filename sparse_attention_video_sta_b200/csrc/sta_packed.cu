// sta_packed.cu -- attention of packed sequences of different lengths, causal
// or not, with grouped heads: the C entry points and the forward kernel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <mutex>

#include "sta_ops.h"

namespace sta {
namespace {

constexpr int kMaxDevices = 64;
__device__ uint32_t g_op_status;  // one word per device: kDevTimeout | kDevBounds
std::mutex g_status_mutex;
uint32_t* g_status_ptr[kMaxDevices] = {};

// Sequence of row t, or -1: the last b with cu[b] <= t, if t is before cu[b + 1].
__device__ int find_sequence(const int32_t* cu, int batch, int t) {
    int lo = 0, hi = batch;  // cu[lo] <= t < cu[hi], if any
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (cu[mid + 1] <= t)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo < batch && cu[lo] <= t ? lo : -1;
}

// One warp for each (query, head): keys one after another, D / 32 elements of
// the head in each lane, running maximum and sum.
template <int D>
__global__ void packed_forward_simple(PackedProblem p, Rows q, Rows k, Rows v, Rows o, float* lse) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
    if (w >= int64_t(p.tokens_q) * p.heads) return;
    const int t = int(w / p.heads), h = int(w % p.heads), hk = h / p.group;
    const int b = find_sequence(p.cu_q, p.batch, t);
    float acc[E] = {}, m = -INFINITY, l = 0.0f;
    if (b < 0 && !p.clear_tail) return;
    if (b >= 0) {
        const int q0 = p.cu_q[b], nq = p.cu_q[b + 1] - q0;
        const int k0 = max(0, min(p.cu_k[b], p.tokens_k)), nk = max(0, min(p.cu_k[b + 1], p.tokens_k) - k0);
        const int vis = p.causal ? min(nk, nk - nq + (t - q0) + 1) : nk;
        float qv[E];
        for (int e = 0; e < E; ++e) qv[e] = __bfloat162float(q.p[t * q.ts + h * q.hs + lane * E + e]);
        for (int j = 0; j < vis; ++j) {
            float s = 0.0f;
            for (int e = 0; e < E; ++e)
                s += qv[e] * __bfloat162float(k.p[int64_t(k0 + j) * k.ts + hk * k.hs + lane * E + e]);
            for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(~0u, s, i);
            s *= p.scale;
            const float mn = fmaxf(m, s), a = expf(m - mn), pr = expf(s - mn);
            for (int e = 0; e < E; ++e)
                acc[e] = acc[e] * a + pr * __bfloat162float(v.p[int64_t(k0 + j) * v.ts + hk * v.hs + lane * E + e]);
            l = l * a + pr;
            m = mn;
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    for (int e = 0; e < E; ++e) o.p[t * o.ts + h * o.hs + lane * E + e] = __float2bfloat16(acc[e] * inv);
    if (lane == 0) lse[int64_t(h) * p.tokens_q + t] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t op_status_word(uint32_t** out) {
    int dev = -1;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_status_mutex);
    if (g_status_ptr[dev] == nullptr) {
        void* p = nullptr;
        if (cudaError_t e = cudaGetSymbolAddress(&p, g_op_status); e != cudaSuccess) return e;
        g_status_ptr[dev] = static_cast<uint32_t*>(p);
    }
    *out = g_status_ptr[dev];
    return cudaSuccess;
}

sta_status packed_problem(const sta_packed* p, bool pointers, PackedProblem* out) {
    if (p == nullptr || p->batch < 0 || p->heads < 1 || p->kv_heads < 1 || p->heads % p->kv_heads != 0 ||
        p->tokens_q < 0 || p->tokens_k < 0 || (p->causal != 0 && p->causal != 1) ||
        (p->clear_tail != 0 && p->clear_tail != 1))
        return STA_ERR_INVALID_ARG;
    if (!std::isfinite(p->softmax_scale) || !(p->softmax_scale > 0.0f)) return STA_ERR_INVALID_ARG;
    if (p->head_dim != 64 && p->head_dim != 128) return STA_ERR_UNSUPPORTED;
    const int32_t group = p->heads / p->kv_heads;
    if (group > 128) return STA_ERR_UNSUPPORTED;
    if (p->tokens_q > INT32_MAX || p->tokens_k > INT32_MAX || (p->tokens_q + 128) * p->heads > INT32_MAX ||
        (p->tokens_k + 128) * p->kv_heads > INT32_MAX ||
        p->batch > (1 << 24))
        return STA_ERR_UNSUPPORTED;
    if (pointers && p->batch > 0) {
        if (p->cu_q == nullptr || p->cu_k == nullptr || reinterpret_cast<uintptr_t>(p->cu_q) % 4 != 0 ||
            reinterpret_cast<uintptr_t>(p->cu_k) % 4 != 0)
            return STA_ERR_INVALID_ARG;
    }
    *out = PackedProblem{p->batch, p->heads, p->kv_heads, group, int32_t(p->tokens_q), int32_t(p->tokens_k),
                         p->cu_q, p->cu_k, p->causal, p->clear_tail, p->softmax_scale, nullptr};
    return STA_OK;
}

cudaError_t launch_packed_forward(const PackedProblem& p, int head_dim, const Rows& q, const Rows& k, const Rows& v,
                                  const Rows& o, float* lse, void*, cudaStream_t stream) {
    const int64_t warps = int64_t(p.tokens_q) * p.heads;
    const unsigned grid = unsigned((warps + 3) / 4);
    if (head_dim == 128)
        packed_forward_simple<128><<<grid, 128, 0, stream>>>(p, q, k, v, o, lse);
    else
        packed_forward_simple<64><<<grid, 128, 0, stream>>>(p, q, k, v, o, lse);
    return cudaGetLastError();
}

}  // namespace sta

using namespace sta;

extern "C" {

sta_status sta_packed_workspace(const sta_packed* p, int32_t backward, int64_t* bytes) {
    PackedProblem pp;
    if (bytes == nullptr || (backward != 0 && backward != 1)) return STA_ERR_INVALID_ARG;
    if (sta_status st = packed_problem(p, false, &pp); st != STA_OK) return st;
    *bytes = 256 + (backward ? int64_t(4) * pp.heads * pp.tokens_q : 0);
    return STA_OK;
}

// Checks of a packed call's buffers: the query-like tensors, then the key-like ones.
static sta_status packed_buffers(const sta_packed* p, bool backward, PackedProblem* pp, const sta_rows* const* rows,
                                 int n_q, int n_k, const void* lse, const void* workspace, int64_t workspace_bytes) {
    if (sta_status st = packed_problem(p, true, pp); st != STA_OK) return st;
    int64_t need = 0;
    if (sta_status st = sta_packed_workspace(p, backward, &need); st != STA_OK) return st;
    for (int i = 0; i < n_q + n_k; ++i)
        if (!rows_ok(rows[i], i < n_q ? p->tokens_q : p->tokens_k)) return STA_ERR_INVALID_ARG;
    if (p->tokens_q > 0 && (lse == nullptr || reinterpret_cast<uintptr_t>(lse) % 4 != 0)) return STA_ERR_INVALID_ARG;
    if (p->tokens_q == 0 && (!backward || p->tokens_k == 0)) return STA_OK;  // nothing to do
    if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || workspace_bytes < need)
        return STA_ERR_INVALID_ARG;
    return STA_OK;
}

sta_status sta_packed_forward(const sta_packed* p, const sta_rows* q, const sta_rows* k, const sta_rows* v,
                              const sta_rows* o, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
    PackedProblem pp;
    const sta_rows* rows[] = {q, o, k, v};
    if (sta_status st = packed_buffers(p, false, &pp, rows, 2, 2, lse, workspace, workspace_bytes); st != STA_OK) return st;
    if (pp.tokens_q == 0) return STA_OK;
    if (cudaError_t e = op_begin(); e != cudaSuccess) return op_cuda_status(e);
    if (cudaError_t e = op_status_word(&pp.status); e != cudaSuccess) return op_cuda_status(e);
    return op_cuda_status(launch_packed_forward(pp, p->head_dim, rows_of(q), rows_of(k), rows_of(v), rows_of(o), lse,
                                                workspace, static_cast<cudaStream_t>(stream)));
}

sta_status sta_packed_backward(const sta_packed* p, const sta_rows* q, const sta_rows* k, const sta_rows* v,
                               const sta_rows* o, const sta_rows* dout, const float* lse, const sta_rows* dq,
                               const sta_rows* dk, const sta_rows* dv, void* workspace, int64_t workspace_bytes,
                               void* stream) {
    PackedProblem pp;
    const sta_rows* rows[] = {q, o, dout, dq, k, v, dk, dv};
    if (sta_status st = packed_buffers(p, true, &pp, rows, 4, 4, lse, workspace, workspace_bytes); st != STA_OK) return st;
    if (pp.tokens_q == 0 && pp.tokens_k == 0) return STA_OK;
    if (cudaError_t e = op_begin(); e != cudaSuccess) return op_cuda_status(e);
    if (cudaError_t e = op_status_word(&pp.status); e != cudaSuccess) return op_cuda_status(e);
    return op_cuda_status(launch_packed_backward(pp, p->head_dim, rows_of(q), rows_of(k), rows_of(v), rows_of(o),
                                                 rows_of(dout), lse, rows_of(dq), rows_of(dk), rows_of(dv), workspace,
                                                 static_cast<cudaStream_t>(stream)));
}

sta_status sta_operator_status(void* stream) {
    if (cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream)); e != cudaSuccess)
        return op_cuda_status(e);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return op_cuda_status(e);
    uint32_t* p = nullptr;
    if (cudaError_t e = op_status_word(&p); e != cudaSuccess) return op_cuda_status(e);
    uint32_t word = 0;
    if (cudaError_t e = cudaMemcpy(&word, p, sizeof word, cudaMemcpyDeviceToHost); e != cudaSuccess)
        return op_cuda_status(e);
    if (word != 0)
        if (cudaError_t e = cudaMemset(p, 0, sizeof word); e != cudaSuccess) return op_cuda_status(e);
    if (word & kDevBounds) return STA_ERR_BOUNDS;
    return word & kDevTimeout ? STA_ERR_TIMEOUT : STA_OK;
}

}  // extern "C"
