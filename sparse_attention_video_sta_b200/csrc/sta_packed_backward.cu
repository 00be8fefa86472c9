// sta_packed_backward.cu -- gradients of the packed attention.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sta_ops.h"

namespace sta {
namespace {

__device__ int sequence_of(const int32_t* cu, int batch, int t) {
    int lo = 0, hi = batch;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (cu[mid + 1] <= t)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo < batch && cu[lo] <= t ? lo : -1;
}

template <int E>
__device__ float dot(const float* a, const __nv_bfloat16* b) {
    float s = 0.0f;
    for (int e = 0; e < E; ++e) s += a[e] * __bfloat162float(b[e]);
    for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(~0u, s, i);
    return s;
}

// One warp for each (query, head): D = dO.O, then dQ over the visible keys.
template <int D>
__global__ void packed_dq_simple(PackedProblem p, Rows q, Rows k, Rows v, Rows o, Rows dout, const float* lse, Rows dq,
                                 float* dsum) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
    if (w >= int64_t(p.tokens_q) * p.heads) return;
    const int t = int(w / p.heads), h = int(w % p.heads), hk = h / p.group;
    const int b = sequence_of(p.cu_q, p.batch, t);
    if (b < 0 && !p.clear_tail) return;
    float acc[E] = {};
    if (b >= 0) {
        const int q0 = p.cu_q[b], nq = p.cu_q[b + 1] - q0;
        const int k0 = max(0, min(p.cu_k[b], p.tokens_k)), nk = max(0, min(p.cu_k[b + 1], p.tokens_k) - k0);
        const int vis = p.causal ? min(nk, nk - nq + (t - q0) + 1) : nk;
        float qv[E], dov[E];
        for (int e = 0; e < E; ++e) {
            qv[e] = __bfloat162float(q.p[t * q.ts + h * q.hs + lane * E + e]);
            dov[e] = __bfloat162float(dout.p[t * dout.ts + h * dout.hs + lane * E + e]);
        }
        const float d = dot<E>(dov, o.p + t * o.ts + h * o.hs + lane * E), ls = lse[int64_t(h) * p.tokens_q + t];
        if (lane == 0) dsum[int64_t(h) * p.tokens_q + t] = d;
        for (int j = 0; j < vis; ++j) {
            const __nv_bfloat16* kj = k.p + int64_t(k0 + j) * k.ts + hk * k.hs + lane * E;
            const __nv_bfloat16* vj = v.p + int64_t(k0 + j) * v.ts + hk * v.hs + lane * E;
            const float ds = expf(p.scale * dot<E>(qv, kj) - ls) * (dot<E>(dov, vj) - d);
            for (int e = 0; e < E; ++e) acc[e] += ds * __bfloat162float(kj[e]);
        }
    }
    for (int e = 0; e < E; ++e) dq.p[t * dq.ts + h * dq.hs + lane * E + e] = __float2bfloat16(p.scale * acc[e]);
}

// One warp for each (key, key head): dK and dV over the queries that see it.
template <int D>
__global__ void packed_dkdv_simple(PackedProblem p, Rows q, Rows k, Rows v, Rows dout, const float* lse,
                                   const float* dsum, Rows dk, Rows dv) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
    if (w >= int64_t(p.tokens_k) * p.kv_heads) return;
    const int t = int(w / p.kv_heads), hk = int(w % p.kv_heads);
    const int b = sequence_of(p.cu_k, p.batch, t);
    if (b < 0 && !p.clear_tail) return;
    float ak[E] = {}, av[E] = {};
    if (b >= 0) {
        const int k0 = p.cu_k[b], nk = p.cu_k[b + 1] - k0;
        const int q0 = max(0, min(p.cu_q[b], p.tokens_q)), nq = max(0, min(p.cu_q[b + 1], p.tokens_q) - q0);
        float kv[E], vv[E];
        for (int e = 0; e < E; ++e) {
            kv[e] = __bfloat162float(k.p[t * k.ts + hk * k.hs + lane * E + e]);
            vv[e] = __bfloat162float(v.p[t * v.ts + hk * v.hs + lane * E + e]);
        }
        for (int i = p.causal ? max(0, (t - k0) - (nk - nq)) : 0; i < nq; ++i)
            for (int h = hk * p.group; h < (hk + 1) * p.group; ++h) {
                const __nv_bfloat16* qi = q.p + int64_t(q0 + i) * q.ts + h * q.hs + lane * E;
                const __nv_bfloat16* di = dout.p + int64_t(q0 + i) * dout.ts + h * dout.hs + lane * E;
                const int64_t r = int64_t(h) * p.tokens_q + q0 + i;
                const float pr = expf(p.scale * dot<E>(kv, qi) - lse[r]), ds = pr * (dot<E>(vv, di) - dsum[r]);
                for (int e = 0; e < E; ++e) {
                    av[e] += pr * __bfloat162float(di[e]);
                    ak[e] += ds * __bfloat162float(qi[e]);
                }
            }
    }
    for (int e = 0; e < E; ++e) {
        dk.p[t * dk.ts + hk * dk.hs + lane * E + e] = __float2bfloat16(p.scale * ak[e]);
        dv.p[t * dv.ts + hk * dv.hs + lane * E + e] = __float2bfloat16(av[e]);
    }
}

}  // namespace

cudaError_t launch_packed_backward(const PackedProblem& p, int head_dim, const Rows& q, const Rows& k, const Rows& v,
                                   const Rows& o, const Rows& dout, const float* lse, const Rows& dq, const Rows& dk,
                                   const Rows& dv, void* workspace, cudaStream_t stream) {
    float* dsum = static_cast<float*>(workspace) + 64;  // within the workspace: heads * tokens_q floats
    const unsigned gq = unsigned((int64_t(p.tokens_q) * p.heads + 3) / 4),
                   gk = unsigned((int64_t(p.tokens_k) * p.kv_heads + 3) / 4);
    if (head_dim == 128) {
        if (gq) packed_dq_simple<128><<<gq, 128, 0, stream>>>(p, q, k, v, o, dout, lse, dq, dsum);
        if (gk) packed_dkdv_simple<128><<<gk, 128, 0, stream>>>(p, q, k, v, dout, lse, dsum, dk, dv);
    } else {
        if (gq) packed_dq_simple<64><<<gq, 128, 0, stream>>>(p, q, k, v, o, dout, lse, dq, dsum);
        if (gk) packed_dkdv_simple<64><<<gk, 128, 0, stream>>>(p, q, k, v, dout, lse, dsum, dk, dv);
    }
    return cudaGetLastError();
}

}  // namespace sta
