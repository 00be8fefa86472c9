// sta_cache_attention.cu -- attention over the 8-bit paged cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sta_ops.cuh"
#include "sta_ops.h"

namespace sta {
namespace {

struct CacheArgs {
    sta_cache c;
    PackedProblem p;
    const int32_t* lengths;
    const int32_t* tables;
    int32_t width;
    int64_t stride;
    Rows q, o;
    float* lse;
};

// One warp for each (query, head), tokens one after another.
template <int D>
__global__ void cache_attention_simple(CacheArgs a) {
    constexpr int E = D / 32;
    const PackedProblem& p = a.p;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
    if (w >= int64_t(p.tokens_q) * p.heads) return;
    const int t = int(w / p.heads), h = int(w % p.heads), hk = h / p.group, bt = a.c.block_tokens;
    int b = t, q0 = t, nq = 1;
    if (p.cu_q != nullptr) {
        int lo = 0, hi = p.batch;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (p.cu_q[mid + 1] <= t)
                lo = mid + 1;
            else
                hi = mid;
        }
        b = lo < p.batch && p.cu_q[lo] <= t ? lo : -1;
        if (b < 0 && !p.clear_tail) return;
        if (b >= 0) {
            q0 = p.cu_q[b];
            nq = p.cu_q[b + 1] - q0;
        }
    }
    float acc[E] = {}, m = -INFINITY, l = 0.0f, qv[E];
    if (b >= 0) {
        const int len = max(0, min(a.lengths[b], a.width * bt));
        if (a.lengths[b] != len && lane == 0) atomicOr(p.status, kDevBounds);
        const int vis = min(len, a.lengths[b] - nq + (t - q0) + 1);
        for (int e = 0; e < E; ++e) qv[e] = __bfloat162float(a.q.p[t * a.q.ts + h * a.q.hs + lane * E + e]);
        for (int j = 0; j < vis; ++j) {
            const int blk = a.tables[b * a.stride + j / bt];
            if (blk < 0 || blk >= a.c.blocks) {
                if (lane == 0) atomicOr(p.status, kDevBounds);
                continue;
            }
            const int64_t at = int64_t(blk) * a.c.kv_heads + hk;
            const uint8_t* kc = static_cast<const uint8_t*>(a.c.k_codes) + (at * bt + j % bt) * D + lane * E;
            const uint8_t* vc = static_cast<const uint8_t*>(a.c.v_codes) + (at * bt + j % bt) * D + lane * E;
            float s = 0.0f;
            for (int e = 0; e < E; ++e) {
                float x, y, z, u;
                ops::e4m3_floats(kc[e], x, y, z, u);
                s += qv[e] * x;
            }
            for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(~0u, s, i);
            s *= p.scale * a.c.k_scales[at];
            const float mn = fmaxf(m, s), f = expf(m - mn), pr = expf(s - mn), vs = a.c.v_scales[at];
            for (int e = 0; e < E; ++e) {
                float x, y, z, u;
                ops::e4m3_floats(vc[e], x, y, z, u);
                acc[e] = acc[e] * f + pr * vs * x;
            }
            l = l * f + pr;
            m = mn;
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    for (int e = 0; e < E; ++e) a.o.p[t * a.o.ts + h * a.o.hs + lane * E + e] = __float2bfloat16(acc[e] * inv);
    if (lane == 0) a.lse[int64_t(h) * p.tokens_q + t] = l == 0.0f ? -INFINITY : m + logf(l);
}

// Checks of the cache and the problem together.
sta_status cache_problem(const sta_cache* c, const sta_packed* p, bool pointers, PackedProblem* out) {
    if (!cache_ok(c) || p == nullptr) return STA_ERR_INVALID_ARG;
    if (!cache_supported(c)) return STA_ERR_UNSUPPORTED;
    sta_packed own = *p;
    own.tokens_k = 0;
    own.causal = 1;
    own.cu_k = nullptr;
    if (sta_status st = packed_problem(&own, false, out); st != STA_OK) return st;
    if (p->kv_heads != c->kv_heads || p->head_dim != c->head_dim) return STA_ERR_INVALID_ARG;
    if (pointers && p->cu_q == nullptr && p->tokens_q != p->batch) return STA_ERR_INVALID_ARG;
    if (pointers && reinterpret_cast<uintptr_t>(p->cu_q) % 4 != 0) return STA_ERR_INVALID_ARG;
    return STA_OK;
}

}  // namespace
}  // namespace sta

using namespace sta;

extern "C" {

sta_status sta_cache_workspace(const sta_cache* c, const sta_packed* p, int64_t* bytes) {
    PackedProblem pp;
    if (bytes == nullptr) return STA_ERR_INVALID_ARG;
    if (sta_status st = cache_problem(c, p, false, &pp); st != STA_OK) return st;
    *bytes = 256;
    return STA_OK;
}

sta_status sta_cache_attention(const sta_cache* c, const sta_packed* p, const int32_t* lengths,
                               const int32_t* block_tables, int32_t table_width, int64_t table_stride,
                               const sta_rows* q, const sta_rows* o, float* lse, void* workspace,
                               int64_t workspace_bytes, void* stream) {
    CacheArgs a{};
    if (sta_status st = cache_problem(c, p, true, &a.p); st != STA_OK) return st;
    if (table_width < 1 || table_stride < table_width) return STA_ERR_INVALID_ARG;
    if (int64_t(table_width) * c->block_tokens > INT32_MAX) return STA_ERR_UNSUPPORTED;
    if (a.p.batch == 0 || a.p.tokens_q == 0) return STA_OK;
    for (const void* x : {(const void*)lengths, (const void*)block_tables, (const void*)lse})
        if (x == nullptr || reinterpret_cast<uintptr_t>(x) % 4 != 0) return STA_ERR_INVALID_ARG;
    if (!rows_ok(q, a.p.tokens_q) || !rows_ok(o, a.p.tokens_q)) return STA_ERR_INVALID_ARG;
    int64_t need = 0;
    if (sta_status st = sta_cache_workspace(c, p, &need); st != STA_OK) return st;
    if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || workspace_bytes < need)
        return STA_ERR_INVALID_ARG;
    if (cudaError_t e = op_begin(); e != cudaSuccess) return op_cuda_status(e);
    if (cudaError_t e = op_status_word(&a.p.status); e != cudaSuccess) return op_cuda_status(e);
    a.c = *c;
    a.lengths = lengths;
    a.tables = block_tables;
    a.width = table_width;
    a.stride = table_stride;
    a.q = rows_of(q);
    a.o = rows_of(o);
    a.lse = lse;
    const unsigned grid = unsigned((int64_t(a.p.tokens_q) * a.p.heads + 3) / 4);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c->head_dim == 128)
        cache_attention_simple<128><<<grid, 128, 0, s>>>(a);
    else
        cache_attention_simple<64><<<grid, 128, 0, s>>>(a);
    return op_cuda_status(cudaGetLastError());
}

}  // extern "C"
