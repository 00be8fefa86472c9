// sta_packed_fwd.cuh -- what the packed forward's two kernels share: parameters, the softmax of
// half a row of scores, and planning in the kernel.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "sta_ops.cuh"
#include "sta_packed.cuh"
#include "sta_ptx.cuh"

namespace sta {
namespace packed_fwd {

using packed::QWork;

constexpr int kItemQ = 4;  // entries of the item queue in shared memory
constexpr int kBoxBytes = 128 * 128;    // 128 rows x 128 bytes

// Small problems need no lists: every load warp finds its (at most kSelfItems) items from the
// bounds itself, worker c of n taking items c, c + n, ...  That saves a launch and its workspace where
// the whole call is a few microseconds.
constexpr int kSelfItems = kItemQ - 1;
constexpr int kSelfBatch = 32;  // one lane of the load warp for each sequence

struct FwdParams {
    packed::View v;
    PackedProblem prob;
    int32_t self;  // no lists
    int32_t kv_heads, group, causal, tokens_q;
    Rows o;
    Rows vals;  // V
    float* lse;
    float scale, scale_log2;
    // The running maximum m of a row that has seen no score above -inf: finite, so that exp2(S c - m c) of such a
    // score is 0 (c = scale_log2), and m or m c at the end of fp32's range (0 would hide scores below -126 / c
    // that come later).
    float nothing_yet;
    uint32_t q_box_bytes;  // bytes of one box of a query block: group * (128 / group) rows of 128 bytes
    uint32_t* status;
    uint64_t timeout_ns;
};

// The chunk of a walk's V from which on its rows need care: those that some row of the block does not
// see.  Within such a chunk (its first key `key`) rows from `dead` on are seen by none, and are zeroed;
// those in [hidden, dead) are seen by some, and lose what is not finite.
__device__ __forceinline__ int32_t first_care(const QWork& q) { return max(0, (max(q.limit0, 0) >> 7) - q.c0); }
__device__ __forceinline__ int dead_from(const QWork& q, int32_t causal, int key) {
    return min(128, max(0, (causal ? min(q.nkeys, q.limit0 + q.ntok - 1) : q.nkeys) - key));
}
__device__ __forceinline__ int hidden_from(const QWork& q, int key) { return max(0, q.limit0 - key); }
// Rows [lo, lo + n) of V, from q.key0, that may have lost something and that a row of the result sees.
__device__ __forceinline__ int lost_seen(const QWork& q, int limit, int& lo) {
    lo = max(max(q.limit0, 0), q.c0 * 128);
    return min(limit, (q.c0 + q.n) * 128) - lo;
}

// Scores of the 64 keys of a half row from index `n` on to -inf.
__device__ __forceinline__ void mask_from(uint32_t (&sr)[64], int n) {
#pragma unroll
    for (int j = 0; j < 64; ++j)
        if (j >= n) sr[j] = 0xff800000u;
}

// P = exp2(S * c - m * c) for one 64-score half row, packed to bf16 pairs; returns
// the fp32 sum of the unrounded values: LSE is their logarithm, to fp32 accuracy.
// (P's rounding to bf16, at most 2^-8 relative, is the operand type of P V.)
__device__ __forceinline__ float softmax_exp64(const uint32_t (&sr)[64], float c, float m, uint32_t (&pk)[32]) {
    const uint64_t c2 = ptx::f2(c, c);
    const uint64_t nmc2 = ptx::f2(-m * c, -m * c);
    uint64_t acc0 = ptx::f2(0.0f, 0.0f), acc1 = acc0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        float x0, x1;
        ptx::f2_split(ptx::f2_fma(ptx::f2(__uint_as_float(sr[2 * j]), __uint_as_float(sr[2 * j + 1])), c2, nmc2), x0, x1);
        const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
        pk[j] = ptx::pack_bf16x2(p0, p1);
        if (j & 1)
            acc1 = ptx::f2_add(acc1, ptx::f2(p0, p1));
        else
            acc0 = ptx::f2_add(acc0, ptx::f2(p0, p1));
    }
    float r0, r1, r2, r3;
    ptx::f2_split(acc0, r0, r1);
    ptx::f2_split(acc1, r2, r3);
    return (r0 + r1) + (r2 + r3);
}

__device__ __forceinline__ float row_max64(const uint32_t (&sr)[64]) {
    float a0 = __uint_as_float(sr[0]), a1 = __uint_as_float(sr[1]);
    float a2 = __uint_as_float(sr[2]), a3 = __uint_as_float(sr[3]);
#pragma unroll
    for (int j = 4; j < 60; j += 8) {
        a0 = ptx::max3(a0, __uint_as_float(sr[j]), __uint_as_float(sr[j + 1]));
        a1 = ptx::max3(a1, __uint_as_float(sr[j + 2]), __uint_as_float(sr[j + 3]));
        a2 = ptx::max3(a2, __uint_as_float(sr[j + 4]), __uint_as_float(sr[j + 5]));
        a3 = ptx::max3(a3, __uint_as_float(sr[j + 6]), __uint_as_float(sr[j + 7]));
    }
    a0 = ptx::max3(a0, __uint_as_float(sr[60]), __uint_as_float(sr[61]));
    a1 = ptx::max3(a1, __uint_as_float(sr[62]), __uint_as_float(sr[63]));
    return ptx::max3(a0, a1, fmaxf(a2, a3));
}

// The items of worker `id` of `ids` from the bounds (one warp): sequence b in lane b, its bounds cut
// to the tensors and made rising as sta_packed_lists.cu does.
__device__ __forceinline__ void self_items(const PackedProblem& p, QWork* items, int32_t id, int32_t ids) {
    const int lane = threadIdx.x & 31, tpb = 128 / p.group;
    auto bounds = [&](const int32_t* cu, int32_t tokens, int32_t& from, int32_t& n) {
        const int32_t c0 = cu[0], c = lane < p.batch ? cu[lane + 1] : INT32_MIN;
        const int32_t start = max(0, min(c0, tokens));
        int32_t h = max(start, min(c, tokens));
        for (int i = 1; i < 32; i <<= 1) {
            const int32_t y = __shfl_up_sync(~0u, h, i);
            if (lane >= i) h = max(h, y);
        }
        const int32_t y = __shfl_up_sync(~0u, h, 1);
        from = lane == 0 ? start : y;
        n = h - from;
        const bool cut = c0 != 0 || (lane < p.batch && c != h);
        if (__any_sync(~0u, cut) && lane == 0 && id == 0) atomicOr(p.status, kDevBounds);
    };
    int32_t q0, nq, key0, nk;
    bounds(p.cu_q, p.tokens_q, q0, nq);
    bounds(p.cu_k, p.tokens_k, key0, nk);
    const int32_t mine = (nq + tpb - 1) / tpb;
    int32_t upto = mine;
    for (int i = 1; i < 32; i <<= 1) {
        const int32_t y = __shfl_up_sync(~0u, upto, i);
        if (lane >= i) upto += y;
    }
    const int32_t blocks = __shfl_sync(~0u, upto, 31), first = upto - mine;
    for (int i = 0; i <= kSelfItems; ++i) {
        const int32_t u = id + i * ids;
        const bool any = i < kSelfItems && u < blocks * p.kv_heads;
        const int32_t e = any ? blocks - 1 - u / p.kv_heads : 0;  // a causal sequence's last blocks are its longest
        const int b = 31 - __clz(__ballot_sync(~0u, first <= e && mine > 0) | 1u);
        const int32_t t = (e - __shfl_sync(~0u, first, b)) * tpb, n = __shfl_sync(~0u, nq, b), m = __shfl_sync(~0u, nk, b);
        QWork w{};
        w.tok0 = __shfl_sync(~0u, q0, b) + t;
        w.ntok = min(tpb, n - t);
        w.key0 = __shfl_sync(~0u, key0, b);
        w.nkeys = m;
        w.limit0 = p.causal ? m - n + t + 1 : m;
        const int32_t sees = p.causal ? min(m, w.limit0 + w.ntok - 1) : m;
        w.n = any ? max(1, (sees + 127) / 128) : -1;
        w.slot = -1;
        w.hk = u % p.kv_heads;
        if (lane == 0) items[i] = w;
        if (!any) break;  // (an end)
    }
    __syncwarp();
}

// Zero the rows of no sequence: behind the last, and before the first (one warp of each CTA).
__device__ __forceinline__ void self_clear(const PackedProblem& p, int head_dim, const Rows& o, float* lse) {
    const int lane = threadIdx.x & 31;
    int32_t last = max(0, min(p.cu_q[lane <= p.batch ? lane : 0], p.tokens_q));
    const int32_t first = __shfl_sync(~0u, last, 0);
    if (p.batch == kSelfBatch) last = max(last, min(p.cu_q[kSelfBatch], p.tokens_q));
    last = __reduce_max_sync(~0u, last);
    const int32_t none = first + p.tokens_q - last, parts = head_dim / 8;
    for (int64_t i = int64_t(blockIdx.x) * 32 + lane; i < int64_t(none) * p.heads * parts; i += int64_t(gridDim.x) * 32) {
        const int64_t row = i / parts;
        const int32_t nth = int32_t(row / p.heads), h = int32_t(row - int64_t(nth) * p.heads);
        const int32_t tok = nth + (nth < first ? 0 : last - first);
        *reinterpret_cast<uint4*>(o.p + tok * o.ts + h * o.hs + (i - row * parts) * 8) = make_uint4(0u, 0u, 0u, 0u);
        if (i == row * parts) lse[int64_t(h) * p.tokens_q + tok] = -INFINITY;
    }
}

// The same pieces for 32 scores, sr[kAt] .. sr[kAt + 31].
template <int kAt>
__device__ __forceinline__ void mask_from32(uint32_t (&sr)[64], int n) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j >= n) sr[kAt + j] = 0xff800000u;
}
template <int kAt>
__device__ __forceinline__ float row_max32(const uint32_t (&sr)[64]) {
    float a0 = __uint_as_float(sr[kAt]), a1 = __uint_as_float(sr[kAt + 1]);
#pragma unroll
    for (int j = 2; j < 30; j += 4) {
        a0 = ptx::max3(a0, __uint_as_float(sr[kAt + j]), __uint_as_float(sr[kAt + j + 1]));
        a1 = ptx::max3(a1, __uint_as_float(sr[kAt + j + 2]), __uint_as_float(sr[kAt + j + 3]));
    }
    return fmaxf(a0, ptx::max3(a1, __uint_as_float(sr[kAt + 30]), __uint_as_float(sr[kAt + 31])));
}
template <int kAt>
__device__ __forceinline__ float softmax_exp32(const uint32_t (&sr)[64], float c, float m, uint32_t (&pk)[32]) {
    const uint64_t c2 = ptx::f2(c, c), nmc2 = ptx::f2(-m * c, -m * c);
    uint64_t acc0 = ptx::f2(0.0f, 0.0f), acc1 = acc0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float x0, x1;
        ptx::f2_split(ptx::f2_fma(ptx::f2(__uint_as_float(sr[kAt + 2 * j]), __uint_as_float(sr[kAt + 2 * j + 1])), c2, nmc2),
                      x0, x1);
        const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
        pk[kAt / 2 + j] = ptx::pack_bf16x2(p0, p1);
        if (j & 1)
            acc1 = ptx::f2_add(acc1, ptx::f2(p0, p1));
        else
            acc0 = ptx::f2_add(acc0, ptx::f2(p0, p1));
    }
    float r0, r1, r2, r3;
    ptx::f2_split(acc0, r0, r1);
    ptx::f2_split(acc1, r2, r3);
    return (r0 + r1) + (r2 + r3);
}

// The kernel for short walks (sta_packed_pair.cu).
cudaError_t launch_forward_pair(int head_dim, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                const FwdParams& fp, int64_t items, int sms, cudaStream_t stream);

}  // namespace packed_fwd
}  // namespace sta
