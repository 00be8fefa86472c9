// sta_cache.cu -- the 8-bit paged cache: writing tokens into it, and the block
// tables and slot maps of a serving step.  (Attention over it: sta_cache_attention.cu.)
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "sta_ops.h"
#include "sta_ops.cuh"
#include "sta_packed.cuh"

namespace sta {

bool cache_ok(const sta_cache* c) {
    if (c == nullptr || c->blocks < 1 || c->kv_heads < 1) return false;
    for (const void* p : {(const void*)c->k_codes, (const void*)c->v_codes})
        if (p == nullptr || reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    for (const void* p : {(const void*)c->k_scales, (const void*)c->v_scales})
        if (p == nullptr || reinterpret_cast<uintptr_t>(p) % 4 != 0) return false;
    return true;
}

bool cache_supported(const sta_cache* c) {
    const int bt = c->block_tokens;
    return (bt == 16 || bt == 32 || bt == 64 || bt == 128) && (c->head_dim == 64 || c->head_dim == 128) &&
           c->kv_heads <= 65535;
}

namespace {

// ---------------------------------------------------------------- append
constexpr int kAppendThreads = 128;

// Exponent e of the smallest power of two 2^e, -60 <= e <= 120, with
// amax <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = int(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, -60), 120);
}

__device__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {  // leaves NaN out
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Codes of 8 values, already divided by their scale.
__device__ uint2 codes8(const float (&x)[8]) {
    return make_uint2(uint32_t(ops::e4m3x2(x[0], x[1])) | uint32_t(ops::e4m3x2(x[2], x[3])) << 16,
                      uint32_t(ops::e4m3x2(x[4], x[5])) | uint32_t(ops::e4m3x2(x[6], x[7])) << 16);
}

// One CTA takes the runs (tokens of one block, next to each other) that begin
// among its `range` tokens, for one head of K or V.  A run's values stay in
// registers between the reduction of their maximum and their rounding, so each
// is read once: 128 threads hold a block of 128 tokens x 128 in 64 registers.
// Bound by HBM: 2 bytes read and 1 written for each value.  22600 prompt tokens, 8 key heads, d = 128
// (139 MB): 27.4 us, 5.1 TB/s.  Instructions count here: the maximum and the scaling on pairs of bf16, one
// multiplication where the scale is a power of two (a division compiled beside it took 10 us), and
// addresses without a lookup where a run's slots follow one another: 45 us before these three.
template <int D, int BT>
__global__ void __launch_bounds__(kAppendThreads, D * BT <= 8192 ? 8 : 4)
cache_append_kernel(sta_cache c, Rows k, Rows v, int64_t tokens, const int64_t* __restrict__ slots, int range,
                    uint32_t* status) {
    constexpr int kPer = D / 8;                          // threads for one token
    constexpr int kStep = kAppendThreads / kPer;         // tokens in one pass
    constexpr int kPasses = BT / kStep > 0 ? BT / kStep : 1;
    constexpr int kMaxRange = kAppendThreads;
    constexpr int kLog2 = BT == 16 ? 4 : BT == 32 ? 5 : BT == 64 ? 6 : 7;
    __shared__ uint32_t sh_first[kAppendThreads / 32];  // tokens of the range that begin a run
    __shared__ int sh_n;
    __shared__ int sh_off[BT + 1];
    __shared__ float sh_max[kAppendThreads / 32];
    __shared__ int64_t sh_slot[kMaxRange + BT + 2];  // of tokens t0 - 1, t0, ...
    const int tid = threadIdx.x, h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const Rows x = is_v ? v : k;
    uint8_t* codes = static_cast<uint8_t*>(is_v ? c.v_codes : c.k_codes);
    float* scales = is_v ? c.v_scales : c.k_scales;
    const int64_t n_slots = int64_t(c.blocks) * BT;
    const int64_t t0 = int64_t(blockIdx.x) * range, t1 = min(t0 + range, tokens);
    ops::grid_launch_dependents();
    ops::grid_wait();
    for (int i = tid; i < range + BT + 2; i += kAppendThreads) {
        const int64_t t = t0 - 1 + i;
        sh_slot[i] = t >= 0 && t < tokens ? slots[t] : -1;
    }
    __syncthreads();
    {
        const int64_t s = tid < t1 - t0 ? sh_slot[tid + 1] : -1, before = sh_slot[tid < range ? tid : 0];
        if (s >= n_slots) atomicOr(status, kDevBounds);
        const uint32_t starts =
            __ballot_sync(~0u, s >= 0 && s < n_slots && !(before >= 0 && before >> kLog2 == s >> kLog2));
        if (tid % 32 == 0) sh_first[tid / 32] = starts;
    }
    __syncthreads();
    for (int word = 0; word < kAppendThreads / 32; ++word)
    for (uint32_t left = sh_first[word]; left != 0u; left &= left - 1) {
        const int64_t t = t0 + word * 32 + __ffs(left) - 1;
        const int64_t* mine = sh_slot + (t - t0 + 1);
        const int64_t blk = mine[0] >> kLog2;
        // ---- the run's length and offsets
        if (tid == 0) sh_n = BT + 1;
        __syncthreads();
        bool odd = false;
        for (int i = tid; i < BT + 1; i += kAppendThreads) {
            const int64_t si = mine[i];
            const bool in = si >> kLog2 == blk;
            sh_off[i] = in ? int(si & (BT - 1)) : -1;
            if (!in) atomicMin(&sh_n, i);
            if (in && i > 0 && si != mine[i - 1] + 1) odd = true;  // (past the run's end this may be said in vain)
        }
        const bool in_order = !__syncthreads_or(odd);
        // (a run longer than a block names slots twice: what is past a block's worth is left out, and reported)
        const int n = min(sh_n, BT);
        if (sh_n > BT && tid == 0) atomicOr(status, kDevBounds);
        const int col = (tid % kPer) * 8, j0 = tid / kPer;
        uint4 raw[kPasses];
        const __nv_bfloat16* src = x.p + (t + j0) * x.ts + h * x.hs + col;
        const int64_t step = kStep * x.ts;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (i * kStep + j0 < n) raw[i] = __ldg(reinterpret_cast<const uint4*>(src + i * step));
        }
        uint32_t top = 0;  // two maxima, of magnitudes in bf16
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
            top = bf16x2_max(top, bf16x2_max(bf16x2_max(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu),
                                             bf16x2_max(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu)));
        float amax = fmaxf(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u));
        for (int i = 16; i > 0; i >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, i));
        if (tid % 32 == 0) sh_max[tid / 32] = amax;
        __syncthreads();
        amax = fmaxf(fmaxf(sh_max[0], sh_max[1]), fmaxf(sh_max[2], sh_max[3]));
        // ---- the block's scale
        const int64_t at = blk * c.kv_heads + h;
        float scale = __uint_as_float(uint32_t(scale_exponent(amax) + 127) << 23);
        uint8_t* page = codes + at * (BT * D);
        if (sh_off[0] != 0) {  // the block holds tokens already
            float old = scales[at];
            if (!(old > 0.0f) || isinf(old)) old = ldexpf(1.0f, -60);
            if (scale > old) {
                const float ratio = old / scale;
                for (int i = tid; i < BT * D / 8; i += kAppendThreads) {
                    uint2 u = reinterpret_cast<uint2*>(page)[i];
                    float y[8];
                    ops::e4m3_floats(u.x, y[0], y[1], y[2], y[3]);
                    ops::e4m3_floats(u.y, y[4], y[5], y[6], y[7]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] *= ratio;
                    reinterpret_cast<uint2*>(page)[i] = codes8(y);
                }
            } else {
                scale = old;
            }
        }
        __syncthreads();  // every thread has read the old scale, and the old codes are rewritten
        if (tid == 0) scales[at] = scale;
        const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0u;
        const float inv = 1.0f / scale;  // exact for a power of two, and then a bf16 as well
        const uint32_t inv2 = (__float_as_uint(inv) >> 16) * 0x10001u;
        auto floats = [](const uint32_t (&w)[4], float (&y)[8]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[2 * e] = __uint_as_float(w[e] << 16);
                y[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            }
        };
        if (pow2 && in_order) {
            uint8_t* dst = page + (sh_off[0] + j0) * D + col;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                // (exact; what falls below bf16's range is 0 in e4m3)
                const uint32_t w[4] = {bf16x2_mul(raw[i].x, inv2), bf16x2_mul(raw[i].y, inv2), bf16x2_mul(raw[i].z, inv2),
                                       bf16x2_mul(raw[i].w, inv2)};
                float y[8];
                floats(w, y);
                if (i * kStep + j0 < n) *reinterpret_cast<uint2*>(dst + i * kStep * D) = codes8(y);
            }
        } else {  // a scale that the caller set, or slots out of order: small code, the values read again
#pragma unroll 1
            for (int j = j0; j < n; j += kStep) {
                bool again = false;  // a slot named twice keeps the later token
                for (int i = j + 1; i < n; ++i) again |= sh_off[i] == sh_off[j];
                if (again) continue;
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + (j - j0) * x.ts));
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                float y[8];
                floats(w, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] /= scale;
                *reinterpret_cast<uint2*>(page + sh_off[j] * D + col) = codes8(y);
            }
        }
        __syncthreads();  // sh_off and sh_n are used again
    }
}

template <int D, int BT>
cudaError_t launch_append(const sta_cache& c, const Rows& k, const Rows& v, int64_t tokens, const int64_t* slots,
                          uint32_t* status, cudaStream_t stream) {
    // One token for each CTA while that is at most some 16 CTAs to an SM: a serving step's
    // tokens are all in blocks of their own.  Else a block's worth, which holds the beginning
    // of one or two runs of a prompt.
    const int range = tokens * c.kv_heads * 2 <= 4096 ? 1 : BT;  // (at most kMaxRange)
    const int64_t gx = (tokens + range - 1) / range;
    if (gx > INT32_MAX) return cudaErrorInvalidValue;
    return packed::launch(cache_append_kernel<D, BT>, dim3(unsigned(gx), unsigned(c.kv_heads), 2), kAppendThreads, 0, stream,
                          true, c, k, v, tokens, slots, range, status);
}

// ---------------------------------------------------------------- extend
constexpr int kExtendThreads = 1024;
constexpr unsigned kExtendCluster = 16;
constexpr int kMaxRequests = 8192;
constexpr int extend_smem(int batch) { return (4 * batch + 3) * int(sizeof(int32_t)); }

struct ExtendParams {
    int32_t batch, bt, bt_log2, width, pool;
    int64_t stride, max_slots;
    const int32_t* add;
    const int32_t* len;
    int32_t* len_out;
    int32_t* tables;
    int32_t* free_blocks;
    const int32_t* count;
    int32_t* count_out;
    int64_t* slots;
    int32_t* cu;
    int32_t* shortage;
};

// Sums of each of `v` over the threads before this one, in place; `total`: over all.
constexpr int kSums = 3;
__device__ void block_scan(int64_t (&v)[kSums], int64_t (*sh)[kSums], int64_t (&total)[kSums]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x[kSums];
#pragma unroll
    for (int k = 0; k < kSums; ++k) x[k] = v[k];
    for (int i = 1; i < 32; i <<= 1)
#pragma unroll
        for (int k = 0; k < kSums; ++k) {
            const int64_t y = __shfl_up_sync(~0u, x[k], i);
            if (lane >= i) x[k] += y;
        }
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < kSums; ++k) sh[warp][k] = x[k];
    __syncthreads();
    // every warp sums the warps' totals for itself
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
        int64_t s = sh[lane][k];
        for (int i = 1; i < 32; i <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, s, i);
            if (lane >= i) s += y;
        }
        total[k] = __shfl_sync(~0u, s, 31);
        const int64_t before = __shfl_sync(~0u, s, warp > 0 ? warp - 1 : 0);
        v[k] = (warp > 0 ? before : 0) + x[k] - v[k];
    }
}

// The last b in [0, n) with cu[b] <= t, for a rising cu with cu[0] <= t (one warp, the same t in all lanes).
__device__ int last_at_most(const int32_t* cu, int n, int32_t t) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
    for (int step = 1024; step > 0; step >>= 5) {  // 32 candidates, `step` apart, at a time; n <= 32 * 1024
        const int b = lo + lane * step;
        lo += (__popc(__ballot_sync(~0u, b < n && cu[b] <= t)) - 1) * step;
    }
    return lo;
}

// `n` entries, entry j by lane j % 32 of a warp: put(j, get(j)), four loads on their way at once.
template <class Get, class Put>
__device__ void each_of(int n, Get get, Put put) {
    for (int j0 = threadIdx.x & 31; j0 < n; j0 += 128) {
        int32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j0 + 32 * i < n) x[i] = get(j0 + 32 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j0 + 32 * i < n) put(j0 + 32 * i, x[i]);
    }
}

// One cluster.  Every CTA sums the requests for itself (new tokens, blocks
// returned, blocks needed) into its own shared memory; then all share the
// pushes, meet, and share the tables and slots.  The reads of `len` and `count`
// come before the cluster's meeting and their writes after it, so the outputs
// may be the inputs.  Latency-bound: one launch in place of a chain of scans (64 requests, one token
// each: 6.8 us a call, nearly all of it the host's; 500 requests with 121000 new tokens: 9.7 us).  Its steps
// are round trips: loads go four at a time, the three sums share their barriers, and a warp
// finds the requests of its 128 slots by ballots (a binary search in each thread: 20 us).
__global__ void __launch_bounds__(kExtendThreads) cache_extend_kernel(const ExtendParams p) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ int32_t sh[];
    __shared__ int64_t sh_scan[32][kSums];
    const int B = p.batch, per = (B + kExtendThreads - 1) / kExtendThreads;
    int32_t* s_len = sh;           // tokens held
    int32_t* s_cu = s_len + B;     // new tokens before this request; [B]: all
    int32_t* s_back = s_cu + B + 1;  // blocks returned before it; [B]: all
    int32_t* s_need = s_back + B + 1;  // blocks needed before it; [B]: all
    const int tid = threadIdx.x, first = tid * per, last = min(first + per, B);
    const int64_t row = int64_t(p.width) * p.bt;  // tokens that a table holds
    ops::grid_launch_dependents();
    ops::grid_wait();
    const int32_t count = *p.count;
    bool bad = count < 0 || count > p.pool;
    int64_t sums[kSums] = {0, 0, 0}, totals[kSums];
    int64_t &add = sums[0], &back = sums[1], &need = sums[2];
    for (int b = first; b < last; ++b) {
        const int64_t n = p.len[b], a = p.add[b];
        if (n < 0 || n > row || n + (a > 0 ? a : 0) > row || n + (a > 0 ? a : 0) > INT32_MAX) bad = true;
        const int64_t held = (n + p.bt - 1) / p.bt;
        s_len[b] = int32_t(n);
        if (a < 0) {
            back += held;
        } else {
            add += a;
            need += (n + a + p.bt - 1) / p.bt - held;
        }
    }
    block_scan(sums, sh_scan, totals);
    int64_t at_add = sums[0], at_back = sums[1], at_need = sums[2];
    const int64_t all_add = totals[0], all_back = totals[1], all_need = totals[2];
    bad = __syncthreads_or(bad) || all_add > p.max_slots || all_add > INT32_MAX || count + all_back > p.pool;
    const int64_t there = count + all_back;
    const int64_t lack = all_need > there ? all_need - there : 0;
    const bool fine = !bad && lack == 0;
    // (sums that do not fit are only read where `fine`)
    for (int b = first; b < last; ++b) {
        const int64_t n = s_len[b], a = p.add[b], held = (n + p.bt - 1) / p.bt;
        s_cu[b] = int32_t(at_add);
        s_back[b] = int32_t(at_back);
        s_need[b] = int32_t(at_need);
        if (a < 0) {
            at_back += held;
        } else {
            at_add += a;
            at_need += (n + a + p.bt - 1) / p.bt - held;
        }
    }
    if (tid == 0) {
        s_cu[B] = int32_t(all_add);
        s_back[B] = int32_t(all_back);
        s_need[B] = int32_t(all_need);
    }
    __syncthreads();
    const int rank = int(cluster.block_rank()), size = int(cluster.num_blocks());
    const int warp = tid / 32, lane = tid % 32, n_warps = kExtendThreads / 32;
    if (fine && all_back > 0)
        for (int b = rank * n_warps + warp; b < B; b += size * n_warps)
            each_of(s_back[b + 1] - s_back[b], [&](int j) { return p.tables[b * p.stride + j]; },
                    [&](int j, int32_t x) { p.free_blocks[count + s_back[b] + j] = x; });
    cluster.sync();  // the stack is whole, and every CTA has read the lengths and the count
    if (fine)
        for (int b = rank * n_warps + warp; b < B; b += size * n_warps) {
            const int held = (s_len[b] + p.bt - 1) / p.bt;
            each_of(s_need[b + 1] - s_need[b], [&](int j) { return p.free_blocks[there - 1 - s_need[b] - j]; },
                    [&](int j, int32_t x) { p.tables[b * p.stride + held + j] = x; });
        }
    const int32_t n_new = fine ? s_cu[B] : 0;
    // a warp takes 128 slots: the requests of its first and last by ballots, those between them in each
    // lane; four entries of the tables on their way at once
    for (int64_t t0 = (rank * n_warps + warp) * 128; t0 < p.max_slots; t0 += size * n_warps * 128) {
        int64_t* out = p.slots + t0 + lane;
        const int room = int(min(p.max_slots - t0, int64_t(128))) - lane;
        const int have = t0 < n_new ? min(n_new - int32_t(t0), 128) : 0, first = int32_t(have > 0 ? t0 : 0);
        int b0 = 0, b1 = 0;
        if (have > 0) {
            b0 = b1 = last_at_most(s_cu, B, first);
            if (s_cu[b0 + 1] < first + have) b1 = last_at_most(s_cu, B, first + have - 1);
        }
        int32_t blk[4], off[4];
        if (b0 == b1) {  // the usual one: all of one request
            const int held = (s_len[b0] + p.bt - 1) >> p.bt_log2, pos0 = s_len[b0] + first - s_cu[b0] + lane;
            const int32_t* table = p.tables + b0 * p.stride;
            const int32_t* popped = p.free_blocks + (there - 1 - s_need[b0]) + held;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = (pos0 + 32 * i) >> p.bt_log2;
                off[i] = (pos0 + 32 * i) & (p.bt - 1);
                blk[i] = lane + 32 * i < have ? *(j < held ? table + j : popped - j) : -1;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = first + lane + 32 * i;
                blk[i] = -1;
                off[i] = 0;
                if (lane + 32 * i < have) {
                    int b = b0, hi = b1;
                    while (b < hi) {
                        const int mid = (b + hi + 1) / 2;
                        if (s_cu[mid] <= t)
                            b = mid;
                        else
                            hi = mid - 1;
                    }
                    const int held = (s_len[b] + p.bt - 1) >> p.bt_log2, pos = s_len[b] + t - s_cu[b], j = pos >> p.bt_log2;
                    blk[i] = j < held ? p.tables[b * p.stride + j] : p.free_blocks[there - 1 - s_need[b] - (j - held)];
                    off[i] = pos & (p.bt - 1);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (32 * i < room) out[32 * i] = uint32_t(blk[i]) < uint32_t(p.pool) ? int64_t(blk[i]) * p.bt + off[i] : -1;
    }
    if (rank == 0) {
        for (int b = tid; b <= B; b += kExtendThreads) p.cu[b] = fine ? s_cu[b] : 0;
        for (int b = tid; b < B; b += kExtendThreads) {
            const bool ended = s_back[b + 1] > s_back[b] || p.add[b] < 0;
            const int32_t n = s_len[b];
            p.len_out[b] = !fine ? n : ended ? 0 : n + (s_cu[b + 1] - s_cu[b]);
        }
        if (tid == 0) {
            *p.count_out = fine ? int32_t(there - all_need) : count;
            *p.shortage = bad ? -1 : int32_t(lack > INT32_MAX ? INT32_MAX : lack);
        }
    }
}

// The kernel's limit on dynamic shared memory belongs to all threads of the process: always the most
// that any call needs, so that none lowers it under another's launch.
cudaError_t extend_most_smem() {
    return cudaFuncSetAttribute(cache_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, extend_smem(kMaxRequests));
}

// A cluster of 16 where the device has one (the SMs of a GPC; 500 requests, 121000 new tokens: 11 us when this was
// chosen, with 8 CTAs 14.6); asked once for each device.  (The kernel's attribute belongs to the device as well.)
cudaError_t extend_cluster(unsigned* ctas) {
    constexpr int kDevices = 64;
    static std::atomic<unsigned> known[kDevices];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    unsigned n = dev < kDevices ? known[dev].load() : 0u;
    if (n == 0) {
        cudaError_t e = extend_most_smem();
        if (e == cudaSuccess) e = cudaFuncSetAttribute(cache_extend_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = *ctas;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(*ctas);
        cfg.blockDim = dim3(kExtendThreads);
        cfg.dynamicSmemBytes = extend_smem(kMaxRequests);  // what is known then holds for every batch
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int fit = 0;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&fit, cache_extend_kernel, &cfg);
        if (e != cudaSuccess) return e;
        n = fit > 0 ? *ctas : 8u;
        if (dev < kDevices) known[dev].store(n);
    }
    *ctas = n;
    return cudaSuccess;
}

}  // namespace
}  // namespace sta

using namespace sta;

extern "C" {

sta_status sta_cache_append(const sta_cache* c, const sta_rows* k, const sta_rows* v, int64_t tokens,
                            const int64_t* slots, void* stream) {
    if (!cache_ok(c) || tokens < 0) return STA_ERR_INVALID_ARG;
    if (!cache_supported(c)) return STA_ERR_UNSUPPORTED;
    if (tokens == 0) return STA_OK;
    if (!rows_ok(k, tokens) || !rows_ok(v, tokens) || slots == nullptr || reinterpret_cast<uintptr_t>(slots) % 8 != 0)
        return STA_ERR_INVALID_ARG;
    if (cudaError_t e = op_begin(); e != cudaSuccess) return op_cuda_status(e);
    uint32_t* status = nullptr;
    if (cudaError_t e = op_status_word(&status); e != cudaSuccess) return op_cuda_status(e);
    const Rows kr = rows_of(k), vr = rows_of(v);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
#define STA_APPEND(D, BT) \
    if (c->head_dim == D && c->block_tokens == BT) e = launch_append<D, BT>(*c, kr, vr, tokens, slots, status, s)
    STA_APPEND(64, 16);
    STA_APPEND(64, 32);
    STA_APPEND(64, 64);
    STA_APPEND(64, 128);
    STA_APPEND(128, 16);
    STA_APPEND(128, 32);
    STA_APPEND(128, 64);
    STA_APPEND(128, 128);
#undef STA_APPEND
    return op_cuda_status(e);
}

sta_status sta_cache_extend(int32_t batch, int32_t block_tokens, const int32_t* new_tokens, const int32_t* lengths,
                            int32_t* lengths_out, int32_t* block_tables, int32_t table_width, int64_t table_stride,
                            int32_t* free_blocks, int32_t pool, const int32_t* free_count, int32_t* free_count_out,
                            int64_t* slots, int64_t max_slots, int32_t* cu_new, int32_t* shortage, void* stream) {
    if (batch < 0 || table_width < 1 || table_stride < table_width || pool < 1 || max_slots < 0 || block_tokens < 1)
        return STA_ERR_INVALID_ARG;
    auto bad = [](const void* p) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % 4 != 0; };
    if (batch > 0 && (bad(new_tokens) || bad(lengths) || bad(lengths_out) || bad(block_tables))) return STA_ERR_INVALID_ARG;
    if (bad(free_blocks) || bad(free_count) || bad(free_count_out) || bad(cu_new) || bad(shortage)) return STA_ERR_INVALID_ARG;
    if (max_slots > 0 && (slots == nullptr || reinterpret_cast<uintptr_t>(slots) % 8 != 0)) return STA_ERR_INVALID_ARG;
    if (batch > kMaxRequests || (block_tokens != 16 && block_tokens != 32 && block_tokens != 64 && block_tokens != 128))
        return STA_ERR_UNSUPPORTED;
    if (cudaError_t e = op_begin(); e != cudaSuccess) return op_cuda_status(e);
    ExtendParams p{batch, block_tokens, block_tokens == 16 ? 4 : block_tokens == 32 ? 5 : block_tokens == 64 ? 6 : 7, table_width, pool, table_stride, max_slots, new_tokens, lengths, lengths_out,
                   block_tables, free_blocks, free_count, free_count_out, slots, cu_new, shortage};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kExtendThreads);
    cfg.dynamicSmemBytes = extend_smem(batch);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    if (cfg.dynamicSmemBytes > 48 * 1024)
        if (cudaError_t e = extend_most_smem(); e != cudaSuccess) return op_cuda_status(e);
    // a serving step's few slots and tables need no second CTA
    unsigned ctas = 1;
    if (max_slots > 8 * kExtendThreads || batch > 4 * kExtendThreads / 32) {
        ctas = kExtendCluster;
        if (cudaError_t e = extend_cluster(&ctas); e != cudaSuccess) return op_cuda_status(e);
    }
    attr[1].val.clusterDim.x = ctas;
    cfg.gridDim = dim3(ctas);
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return op_cuda_status(cudaLaunchKernelEx(&cfg, cache_extend_kernel, p));
}

}  // extern "C"
