// sta_packed_backward.cu -- gradients of the packed attention (sta_packed.cu).
//
//   P_ij = exp(scale q_i.k_j - LSE_i),  D_i = dO_i.O_i,  dS_ij = P_ij (dO_i.v_j - D_i),
//   dQ_i = scale sum_j dS_ij k_j,  dK_j = scale sum_i dS_ij q_i,  dV_j = sum_i P_ij dO_i,
// the sums over i running over the queries of every head that shares the key head.
//
// Four launches, no atomics on results: the work lists (sta_packed_lists.cu);
// packed_prep_kernel, -D and -LSE log2(e) of every row of every query block;
// packed_dq_kernel, one query block per item, walking key chunks; packed_dkdv_kernel,
// one key block per item, walking the query blocks that see it.  Query blocks hold the
// rows of all the query heads of a key head (sta_packed.cuh), so dK and dV of a shared
// head are ordinary sums over a block's rows, in the tensor core's fp32 accumulator.
// Both main kernels are the video backward's pipeline (one TMA warp, one tcgen05
// issuing thread, two elementwise warpgroups) with masks.
//
// Masks and rows that are not there.  In a masked chunk P and dS are selected to 0,
// whatever the products held.  Rows of an operand that a product sums over must be
// finite as well, since 0 x inf is not 0: K rows that no query of the block sees (dQ)
// and Q, dO rows behind a block's last token (dK, dV) are overwritten with zeros in
// shared memory by the elementwise warps, once the products that only need the other
// rows have read them; on the causal diagonal the rows that only some see lose what is
// not finite, and the results that see them get it back (scrub_rows, restore).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sta_ops.cuh"
#include "sta_ops.h"
#include "sta_packed.cuh"
#include "sta_ptx.cuh"
#include "sta_wait.cuh"

namespace sta {
namespace {

using packed::KBlock;
using packed::KWork;
using packed::QBlock;
using packed::QWork;

// Warps 0-15 elementwise: four to an SM sub-partition, 32 columns of a row to a thread (8 warps of 64
// columns cover less of a step's round trips: six sequences of 342-2047 tokens, 16 / 2 heads, d = 64, forward
// and backward 171 us against 168); 16 load, 17 MMA.
constexpr int kEwWarps = 16;
constexpr int kEwThreads = kEwWarps * 32;
constexpr int kParts = kEwWarps / 4;  // of a row's 128 columns
constexpr int kLoadWarp = kEwWarps;
constexpr int kMmaWarp = kEwWarps + 1;
constexpr int kThreads = kEwThreads + 64;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kBoxBytes = 128 * 128;  // 128 rows x 128 bytes (64 bf16)
constexpr int kItemQ = 4;
constexpr int kItemConsumers = 1 + kEwWarps;
// At least this much shared memory at launch, so that a CTA has its SM alone (a
// second one would wait in tcgen05.alloc for the first one's 512 columns).
constexpr int kMinSmem = 120 * 1024;
constexpr int smem_launch(int bytes) { return bytes > kMinSmem ? bytes : kMinSmem; }

struct BwdParams {
    packed::View v;
    int32_t kv_heads, group, causal;
    const float* neg_l;  // [query blocks][kv_heads][128]: -LSE log2(e); -inf: no such row, or it sees no key
    float* neg_d;        // the same for -D (the dQ kernel sharpens those of one-chunk walks)
    Rows out_a;          // dQ, or dK
    Rows out_b;          // dV
    float scale, scale_log2;
    uint32_t q_box_bytes;
    uint32_t* status;
    uint64_t timeout_ns;
    int32_t inject;        // debug: the load thread's first wait runs out
    Rows q, k, dout;
};

__device__ __forceinline__ bool wait_bw(uint32_t bar, uint32_t parity, volatile int* abort_flag, const BwdParams& p) {
    return wait_bar_limited(bar, parity, abort_flag, p.status, p.timeout_ns);
}

template <int D>
__device__ __forceinline__ void load_block(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t head, int32_t tok) {
#pragma unroll
    for (int cb = 0; cb < D / 64; ++cb) ops::tma_load_3d(dst + cb * kBoxBytes, m, bar, cb * 64, head, tok);
}

// The item queue.  A CTA's first item is its own number, the others come from a counter; an item
// is only taken when the copies of the one before are issued, so that longest-first levels the CTAs.
template <class Work>
__device__ __forceinline__ bool put_item(uint32_t k, Work& w, const Work* walks, int32_t* next, int32_t n_items, int32_t heads,
                                         uint32_t full0, uint32_t empty0, Work* q, volatile int* abort_flag,
                                         const BwdParams& p) {
    const int32_t u = k == 0 ? int32_t(blockIdx.x) : int32_t(gridDim.x) + atomicAdd(next, 1);
    w.n = -1;
    if (u < n_items) {
        w = walks[u / heads];
        w.hk = u % heads;
    }
    const uint32_t e = k % kItemQ;
    if (k >= uint32_t(kItemQ) && !wait_bw(empty0 + 8u * e, ((k / kItemQ) - 1) & 1u, abort_flag, p)) return false;
    q[e] = w;
    ptx::mbar_arrive(full0 + 8u * e);
    return w.n >= 0;
}
template <class Work>
__device__ __forceinline__ bool get_item(uint32_t k, uint32_t full0, const Work* q, volatile int* abort_flag,
                                        const BwdParams& p, Work& w) {
    if (!wait_bw(full0 + 8u * (k % kItemQ), (k / kItemQ) & 1u, abort_flag, p)) return false;
    w = q[k % kItemQ];
    return true;
}

// 32 fp32 TMEM columns of this thread's lane, times `mul`, as bf16 to dst; `zero`: zeros
// instead.  Every lane loads (the access is warp-wide); lanes with `store` write.
// `fix(r)` changes them before.
template <class Fix>
__device__ __forceinline__ void store_cols(uint32_t taddr, float mul, __nv_bfloat16* dst, bool store, bool zero, Fix&& fix) {
    uint4* d4 = reinterpret_cast<uint4*>(dst);
    uint32_t r[32];
    ptx::tmem_ld32(taddr, r);
    if (!store) return;
    fix(r);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint4 v;
        v.x = ptx::pack_bf16x2(__uint_as_float(r[8 * j + 0]) * mul, __uint_as_float(r[8 * j + 1]) * mul);
        v.y = ptx::pack_bf16x2(__uint_as_float(r[8 * j + 2]) * mul, __uint_as_float(r[8 * j + 3]) * mul);
        v.z = ptx::pack_bf16x2(__uint_as_float(r[8 * j + 4]) * mul, __uint_as_float(r[8 * j + 5]) * mul);
        v.w = ptx::pack_bf16x2(__uint_as_float(r[8 * j + 6]) * mul, __uint_as_float(r[8 * j + 7]) * mul);
        d4[j] = zero ? make_uint4(0u, 0u, 0u, 0u) : v;
    }
}

// 32 columns of zeros.
__device__ __forceinline__ void zero_cols(__nv_bfloat16* dst) {
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<uint4*>(dst)[j] = make_uint4(0u, 0u, 0u, 0u);
}

// As store_cols, but fp32 as they are: a part's sums, four columns of all rows after four columns (a warp's
// stores are whole lines).  `dst`: the part's four columns that `taddr` begins with, this thread's row.
template <class Fix>
__device__ __forceinline__ void store_part(uint32_t taddr, float4* dst, bool store, Fix&& fix) {
    uint32_t r[32];
    ptx::tmem_ld32(taddr, r);
    if (!store) return;
    fix(r);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        dst[j * 128] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]), __uint_as_float(r[4 * j + 2]),
                                   __uint_as_float(r[4 * j + 3]));
}

// A-operand column of K-step kk of a bf16 matrix that the elementwise warpgroups wrote into
// TMEM: warpgroup h packs its 32 columns into columns [32 h, 32 h + 16).
__device__ __forceinline__ uint32_t a_col(int kk) { return uint32_t((kk >> 1) * 32 + (kk & 1) * 8); }

// Rows [from, 128) of a 128-row block in shared memory to zero (128-byte rows in D / 64 boxes;
// the swizzle permutes within rows), by the elementwise threads, visible to tcgen05.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* blk, int from, int thread) {
    for (int i = from * 8 + thread; i < 128 * 8; i += kEwThreads)
#pragma unroll
        for (int cb = 0; cb < D / 64; ++cb)
            *reinterpret_cast<uint4*>(blk + cb * kBoxBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
}

// ---------------------------------------------------------------- prep
// -D and -LSE log2(e) of the rows of every (query block, key head): D / 8 threads for a
// row, 16 bytes of O and dO each.  HBM-bound: O and dO once (8192 tokens, 24 heads, d = 128: 28 us,
// 3.6 TB/s).
template <int D>
__global__ void __launch_bounds__(256) packed_prep_kernel(const PackedProblem p, const packed::View v, Rows o, Rows dout,
                                                          const float* lse, float* neg_l, float* neg_d) {
    constexpr int kTpr = D / 8;
    ops::grid_wait();
    ops::grid_launch_dependents();
    const int part = threadIdx.x % kTpr;
    const int64_t n = int64_t(v.lists->n_q) * p.kv_heads;
    for (int64_t w = blockIdx.x; w < n; w += gridDim.x) {
        const QBlock q = v.qblocks[w / p.kv_heads];
        const int hk = int(w % p.kv_heads);
#pragma unroll
        for (int r0 = 0; r0 < 128; r0 += 256 / kTpr) {
            const int r = r0 + threadIdx.x / kTpr, t = r / p.group, h = hk * p.group + r - t * p.group;
            const bool real = t < q.ntok;
            float acc = 0.0f;
            if (real) {
                const int64_t tok = q.tok0 + t;
                const uint4 a = __ldg(reinterpret_cast<const uint4*>(o.p + tok * o.ts + h * o.hs) + part);
                const uint4 b = __ldg(reinterpret_cast<const uint4*>(dout.p + tok * dout.ts + h * dout.hs) + part);
                const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc = fmaf(__uint_as_float(aw[i] << 16), __uint_as_float(bw[i] << 16), acc);
                    acc = fmaf(__uint_as_float(aw[i] & 0xffff0000u), __uint_as_float(bw[i] & 0xffff0000u), acc);
                }
            }
#pragma unroll
            for (int s = kTpr / 2; s > 0; s >>= 1) acc += __shfl_xor_sync(~0u, acc, s);
            if (part == 0) {
                const float l = real ? lse[int64_t(h) * p.tokens_q + q.tok0 + t] : -INFINITY;
                neg_d[w * 128 + r] = real ? -acc : 0.0f;
                neg_l[w * 128 + r] = l == -INFINITY ? -INFINITY : -l * kLog2e;
            }
        }
    }
}

// ---------------------------------------------------------------- dQ
// Three products for each chunk (S, dP, dQ).  8192 causal tokens, 24 / 8 heads, d = 128: 563 us under a
// profiler, 1.10 PFLOP/s of products, tensor pipe active 58 %; the rest is the chain dP -> dS -> dQ of a chunk,
// since TMEM holds two S but one dP beside dQ.
template <int D>
struct DqCfg {
    static constexpr int kBlk = 128 * D * 2;
    static constexpr int kKStages = 3, kVStages = 2;
    static constexpr int kQOff = 0, kDOOff = kBlk;
    static constexpr int kKOff = 2 * kBlk;
    static constexpr int kVOff = kKOff + kKStages * kBlk;
    static constexpr int kBarOff = kVOff + kVStages * kBlk;
    // k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], q_full, q_empty,
    // s_full[2], dp_full, ds_full, dq_full, drain, item_full[Q], item_empty[Q]
    static constexpr int kNumBars = 2 * kKStages + 2 * kVStages + 8 + 2 * kItemQ;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kQueueOff = kMiscOff + 16;
    static constexpr int kLostOff = kQueueOff + kItemQ * int(sizeof(QWork));  // kLostWords
    static constexpr int kSmemBytes = kLostOff + 4 * packed::kLostWords + 1024;
    static_assert(kQueueOff % 16 == 0, "queue entries are 16-byte aligned");
    static constexpr uint32_t kColS0 = 0, kColDP = 256, kColDQ = 384;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
    static_assert(kColDQ + D <= kTmemCols, "TMEM budget");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
packed_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                 const BwdParams p) {
    using C = DqCfg<D>;
    constexpr int KS = C::kKStages, VS = C::kVStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const uint32_t bar0 = base + C::kBarOff;
    auto k_full = [&](int r) { return bar0 + 8u * r; };
    auto k_empty = [&](int r) { return bar0 + 8u * (KS + r); };
    auto v_full = [&](int r) { return bar0 + 8u * (2 * KS + r); };
    auto v_empty = [&](int r) { return bar0 + 8u * (2 * KS + VS + r); };
    const uint32_t xb = bar0 + 8u * (2 * KS + 2 * VS);
    const uint32_t q_full = xb, q_empty = xb + 8;
    auto s_full = [&](int b) { return xb + 16 + 8u * b; };
    const uint32_t dp_full = xb + 32, ds_full = xb + 40, dq_full = xb + 48, drain = xb + 56;
    const uint32_t item_full0 = xb + 64, item_empty0 = xb + 64 + 8 * kItemQ;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    volatile uint32_t* lost = reinterpret_cast<volatile uint32_t*>(smem + C::kLostOff);
    QWork* item_q = reinterpret_cast<QWork*>(smem + C::kQueueOff);

    if (threadIdx.x == 0) {
        for (int r = 0; r < KS; ++r) {
            ptx::mbar_init(k_full(r), 1);
            ptx::mbar_init(k_empty(r), 1);
        }
        for (int r = 0; r < VS; ++r) {
            ptx::mbar_init(v_full(r), 1);
            ptx::mbar_init(v_empty(r), 1);
        }
        ptx::mbar_init(q_full, 1);
        ptx::mbar_init(q_empty, 1);
        ptx::mbar_init(s_full(0), 1);
        ptx::mbar_init(s_full(1), 1);
        ptx::mbar_init(dp_full, 1);
        ptx::mbar_init(ds_full, kEwWarps);
        ptx::mbar_init(dq_full, 1);
        ptx::mbar_init(drain, 1);
        for (int q = 0; q < kItemQ; ++q) {
            ptx::mbar_init(item_full0 + 8u * q, 1);
            ptx::mbar_init(item_empty0 + 8u * q, kItemConsumers);
        }
        *abort_flag = 0;
        for (int i = 0; i < packed::kLostWords; ++i) lost[i] = 0;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == kLoadWarp && lane == 0) {
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
        ptx::prefetch_tensormap(&tm_do);
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
        ptx::tmem_relinquish();
    }
    ops::grid_wait();  // the lists and the rows' constants
    ops::grid_launch_dependents();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int32_t K = p.kv_heads;

    if (warp == kLoadWarp) {
        if (lane == 0) {
            // ------------------------------------------------------------ load
            const int32_t n_items = p.v.lists->w_q * K;
            uint32_t kit = 0, vit = 0, qc = 0;
            bool ok = !p.inject || wait_bw(drain, 0, abort_flag, p);  // (arrived at on the way out only)
            for (uint32_t kq = 0; ok; ++kq) {
                QWork q;
                if (!put_item(kq, q, p.v.qwalks, &p.v.lists->next_dq, n_items, K, item_full0, item_empty0, item_q, abort_flag, p))
                    break;
                const int32_t hk = q.hk;
                if (!wait_bw(q_empty, (qc & 1u) ^ 1u, abort_flag, p)) break;
                ptx::mbar_arrive_expect_tx(q_full, 2 * (D / 64) * p.q_box_bytes);
                load_block<D>(base + C::kQOff, &tm_q, q_full, hk * p.group, q.tok0);
                load_block<D>(base + C::kDOOff, &tm_do, q_full, hk * p.group, q.tok0);
                ++qc;
                for (int32_t c = q.c0; c < q.c0 + q.n; ++c) {
                    const int rk = int(kit % KS);
                    if (kit >= uint32_t(KS) && !wait_bw(k_empty(rk), ((kit / KS) - 1) & 1u, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    ptx::mbar_arrive_expect_tx(k_full(rk), C::kBlk);
                    load_block<D>(base + C::kKOff + rk * C::kBlk, &tm_k, k_full(rk), hk, q.key0 + c * 128);
                    ++kit;
                    const int rv = int(vit % VS);
                    if (vit >= uint32_t(VS) && !wait_bw(v_empty(rv), ((vit / VS) - 1) & 1u, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    ptx::mbar_arrive_expect_tx(v_full(rv), C::kBlk);
                    load_block<D>(base + C::kVOff + rv * C::kBlk, &tm_v, v_full(rv), hk, q.key0 + c * 128);
                    ++vit;
                }
            }
            // Drain the copies still in flight.
            for (uint32_t it = kit > uint32_t(KS) ? kit - KS : 0u; it < kit; ++it)
                drain_bar(k_full(int(it % KS)), (it / KS) & 1u, p.timeout_ns);
            for (uint32_t it = vit > uint32_t(VS) ? vit - VS : 0u; it < vit; ++it)
                drain_bar(v_full(int(it % VS)), (it / VS) & 1u, p.timeout_ns);
            if (qc > 0) drain_bar(q_full, (qc - 1) & 1u, p.timeout_ns);
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            // ------------------------------------------------------------- MMA
            constexpr uint32_t idesc_s = ptx::idesc_bf16(128, 128, false);
            constexpr uint32_t idesc_dq = ptx::idesc_bf16(128, D, true);
            const uint32_t qaddr = base + C::kQOff, doaddr = base + C::kDOOff;
            uint32_t kbase = 0, gs = 0, qc = 0;
            bool ok = true;
            for (uint32_t kq = 0; ok; ++kq) {
                QWork q;
                if (!get_item(kq, item_full0, item_q, abort_flag, p, q)) break;
                ptx::mbar_arrive(item_empty0 + 8u * (kq % kItemQ));
                if (q.n < 0) break;
                const int32_t n = q.n;
                if (!wait_bw(q_full, qc & 1u, abort_flag, p)) break;
                ++qc;
                ptx::tc_fence_after();
                // S_j = Q K_j^T into S buffer (gs + j) & 1
                auto issue_s = [&](int32_t j) -> bool {
                    const uint32_t it = kbase + uint32_t(j);
                    if (!wait_bw(k_full(int(it % KS)), (it / KS) & 1u, abort_flag, p)) return false;
                    ptx::tc_fence_after();
                    const uint32_t kaddr = base + C::kKOff + (it % KS) * C::kBlk;
                    const uint32_t tS = tmem + C::kColS0 + ((gs + uint32_t(j)) & 1u) * 128u;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t coff = (kk >> 2) * kBoxBytes + (kk & 3) * 32;
                        ptx::mma_ss(tS, ptx::desc_k_sw128(qaddr + coff), ptx::desc_k_sw128(kaddr + coff), idesc_s,
                                    kk > 0 ? 1u : 0u);
                    }
                    ptx::mma_commit(s_full(int((gs + uint32_t(j)) & 1u)));
                    return true;
                };
                // dP_j = dO V_j^T; V_j is then free
                auto issue_dp = [&](int32_t j) -> bool {
                    const uint32_t it = kbase + uint32_t(j);
                    if (!wait_bw(v_full(int(it % VS)), (it / VS) & 1u, abort_flag, p)) return false;
                    ptx::tc_fence_after();
                    const uint32_t vaddr = base + C::kVOff + (it % VS) * C::kBlk;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t coff = (kk >> 2) * kBoxBytes + (kk & 3) * 32;
                        ptx::mma_ss(tmem + C::kColDP, ptx::desc_k_sw128(doaddr + coff), ptx::desc_k_sw128(vaddr + coff),
                                    idesc_s, kk > 0 ? 1u : 0u);
                    }
                    ptx::mma_commit(dp_full);
                    ptx::mma_commit(v_empty(int(it % VS)));
                    return true;
                };
                ok = issue_s(0) && issue_dp(0) && (n < 2 || issue_s(1));
                for (int32_t j = 0; ok && j < n; ++j) {
                    if (!wait_bw(ds_full, (gs + uint32_t(j)) & 1u, abort_flag, p)) { ok = false; break; }
                    ptx::tc_fence_after();
                    // dQ += dS_j K_j (dS from TMEM over dP; K_j MN-major)
                    const uint32_t it = kbase + uint32_t(j);
                    const uint32_t kaddr = base + C::kKOff + (it % KS) * C::kBlk;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        ptx::mma_ts(tmem + C::kColDQ, tmem + C::kColDP + a_col(kk),
                                    ptx::desc_mn_sw128(kaddr + kk * 16 * 128, kBoxBytes), idesc_dq,
                                    (j > 0 || kk > 0) ? 1u : 0u);
                    ptx::mma_commit(k_empty(int(it % KS)));
                    // in issue order after dQ_j, which reads the dS this dP overwrites
                    if (j + 1 < n && !issue_dp(j + 1)) { ok = false; break; }
                    if (j + 2 < n && !issue_s(j + 2)) { ok = false; break; }
                }
                if (!ok) break;
                ptx::mma_commit(dq_full);
                ptx::mma_commit(q_empty);
                kbase += uint32_t(n);
                gs += uint32_t(n);
            }
            ptx::mma_commit(drain);
            drain_bar(drain, 0, p.timeout_ns);
        }
    } else {
        // ------------------------------------------------------- elementwise
        const int h = warp >> 2;  // which 32 columns
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = uint32_t((warp & 3) * 32) << 16;
        const uint64_t c2 = ptx::f2(p.scale_log2, p.scale_log2);
        const int r_tok = row / p.group, r_head = row - r_tok * p.group;
        const uint32_t rows_bar = 1u + uint32_t(warp & 3);  // named barrier of the kParts warps with the same rows
        // [kParts][128 rows], over the query block: S and dP have read it where this is used, and the next one
        // is copied in after dQ
        float* xch = reinterpret_cast<float*>(smem + C::kQOff);
        uint32_t gs = 0, dqc = 0;
        bool ok = true;
        for (uint32_t kq = 0; ok; ++kq) {
            QWork q;
            q.n = -1;
            const bool took = __all_sync(~0u, get_item(kq, item_full0, item_q, abort_flag, p, q));
            __syncwarp();
            if (took && lane == 0) ptx::mbar_arrive(item_empty0 + 8u * (kq % kItemQ));
            if (ptx::bar_red_or(rows_bar, 32 * kParts, !took)) break;  // leave together: they meet again below
            if (q.n < 0) break;
            const int32_t hk = q.hk, n = q.n;
            const bool real = r_tok < q.ntok;
            const int limit = real ? min(q.nkeys, q.limit0 + (p.causal ? r_tok : 0)) : INT32_MAX;
            const int warp_limit = __reduce_min_sync(~0u, limit);
            const int64_t grow = (int64_t(q.block) * K + hk) * 128 + row;
            const float nl = p.neg_l[grow];
            float nd = p.neg_d[grow];
            const uint64_t nl2 = ptx::f2(nl, nl);
            // A walk of one chunk has all of the row's P and dP here, so D = sum P dP is taken from them:
            // dO.O carries O's rounding to bf16 into every dS of the row, which shows (a sixth of the
            // error of dQ and dK at 2048 causal tokens) where a row has few keys; over more keys it
            // averages out.
            const bool exact = n == 1 && q.c0 == 0 && q.slot < 0;
            for (int32_t j = 0; j < n; ++j) {
                const uint32_t step = gs + uint32_t(j);
                // (in an exact walk the warps of the same rows meet at their barrier, whatever failed)
                bool good = __all_sync(~0u, wait_bw(s_full(int(step & 1u)), (step >> 1) & 1u, abort_flag, p));
                if (!good && !exact) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const int key = (q.c0 + j) * 128;  // the chunk's first
                const int seen = limit - (key + 32 * h);  // keys of this part that the row sees
                const bool masked = warp_limit < key + 32 * h + 32;
                if (key + 128 > q.limit0) {  // keys that some row does not see: S has read K, dQ has not
                    if (!wait_bw(k_full(int(step % KS)), (step / KS) & 1u, abort_flag, p)) good = false;  // (has been)
                    uint8_t* kblk = smem + C::kKOff + (step % KS) * C::kBlk;
                    const int dead = min(128, max(0, (p.causal ? min(q.nkeys, q.limit0 + q.ntok - 1) : q.nkeys) - key));
                    if (packed::scrub_rows<D / 64>(kblk, kBoxBytes, max(0, q.limit0 - key), dead, threadIdx.x, kEwThreads))
                        lost[kq % packed::kLostWords] = kq + 1;
                    zero_rows<D>(kblk, dead, threadIdx.x);
                }
                float pr[32];
                {
                    uint32_t sr[32];
                    ptx::tmem_ld32(tmem + lane_addr + C::kColS0 + (step & 1u) * 128u + 32u * h, sr);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x0, x1;
                        ptx::f2_split(ptx::f2_fma(ptx::f2(__uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1])),
                                                  c2, nl2),
                                      x0, x1);
                        pr[2 * i] = ptx::ex2(x0);
                        pr[2 * i + 1] = ptx::ex2(x1);
                    }
                }
                good = good && __all_sync(~0u, wait_bw(dp_full, step & 1u, abort_flag, p));
                if (!good && !exact) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t tdp = tmem + lane_addr + C::kColDP + 32u * h;
                uint32_t pk[16];
                {
                    uint32_t dr[32];
                    ptx::tmem_ld32(tdp, dr);
                    if (masked)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i >= seen) {
                                pr[i] = 0.0f;
                                dr[i] = 0u;
                            }
                    if (exact) {
                        uint64_t a0 = ptx::f2(0.0f, 0.0f), a1 = a0;
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            a0 = ptx::f2_fma(ptx::f2(pr[2 * i], pr[2 * i + 1]),
                                             ptx::f2(__uint_as_float(dr[2 * i]), __uint_as_float(dr[2 * i + 1])), a0);
                            a1 = ptx::f2_fma(ptx::f2(pr[2 * i + 2], pr[2 * i + 3]),
                                             ptx::f2(__uint_as_float(dr[2 * i + 2]), __uint_as_float(dr[2 * i + 3])), a1);
                        }
                        float x0, x1;
                        ptx::f2_split(ptx::f2_add(a0, a1), x0, x1);
                        xch[h * 128 + row] = x0 + x1;
                        if (ptx::bar_red_or(rows_bar, 32 * kParts, !good)) {
                            ok = false;
                            break;
                        }
                        nd = -((xch[row] + xch[128 + row]) + (xch[256 + row] + xch[384 + row]));
                        if (h == 0 && real) p.neg_d[grow] = nd;  // for dK / dV
                        ptx::fence_proxy_async_smem();
                    }
                    const uint64_t nd2 = ptx::f2(nd, nd);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float t0, t1;
                        ptx::f2_split(ptx::f2_mul(ptx::f2(pr[2 * i], pr[2 * i + 1]),
                                                  ptx::f2_add(ptx::f2(__uint_as_float(dr[2 * i]),
                                                                      __uint_as_float(dr[2 * i + 1])),
                                                              nd2)),
                                      t0, t1);
                        pk[i] = ptx::pack_bf16x2(t0, t1);
                    }
                }
                ops::tmem_st16(tdp, pk);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ds_full);
            }
            if (!ok) break;
            if (!__all_sync(~0u, wait_bw(dq_full, dqc & 1u, abort_flag, p))) break;
            ++dqc;
            ptx::tc_fence_after();
            const bool fix = lost[kq % packed::kLostWords] == kq + 1;
            const int lo = max(max(q.limit0, 0), q.c0 * 128), seen = min(limit, (q.c0 + n) * 128) - lo;
            if (h < D / 32) {  // 32 of the D columns for each warpgroup
                auto put_back = [&](uint32_t (&r)[32]) {
                    if (fix)
                        packed::restore(r, p.k.p + (q.key0 + int64_t(lo)) * p.k.ts + hk * p.k.hs + 32 * h, p.k.ts, seen);
                };
                const uint32_t t_dq = tmem + lane_addr + C::kColDQ + 32u * h;
                if (q.slot >= 0)
                    store_part(t_dq, reinterpret_cast<float4*>(p.v.parts + (int64_t(q.slot) * K + hk) * (128 * D)) + 8 * h * 128 + row,
                               real, put_back);
                else
                    store_cols(t_dq, p.scale,
                               p.out_a.p + int64_t(q.tok0 + r_tok) * p.out_a.ts + (hk * p.group + r_head) * p.out_a.hs + 32 * h,
                               real, limit <= 0, put_back);
            }
            ptx::tc_fence_before();
            gs += uint32_t(n);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- dK / dV
// Four products for each query block (S^T, dP^T, dV, dK).  8192 causal tokens, 24 / 8 heads, d = 128:
// 743 us under a profiler, 1.11 PFLOP/s of products, tensor pipe active 58 %; S^T, dP^T, dV and dK fill TMEM, so a
// block's exponentials wait for its scores, which wait for the P of the block before to be read (with eight
// elementwise warps 1650 and 750 of a step's 3550 cycles).
template <int D>
struct DkvCfg {
    static constexpr int kBlk = 128 * D * 2;
    static constexpr int kStages = 2;
    static constexpr int kKOff = 0, kVOff = kBlk;
    // stage: Q block, dO block, -LSE log2(e) [128], -D [128]
    static constexpr int kStQ = 0, kStDO = kBlk, kStL = 2 * kBlk, kStD = 2 * kBlk + 512;
    static constexpr int kStageBytes = 2 * kBlk + 1024;
    static constexpr int kStageOff = 2 * kBlk;
    static constexpr int kBarOff = kStageOff + kStages * kStageBytes;
    // st_full[2], st_empty[2], kv_full, kv_empty, s_full, dp_full, p_full,
    // ds_full, dkv_full, drain, item_full[Q], item_empty[Q]
    static constexpr int kNumBars = 2 * kStages + 8 + 2 * kItemQ;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kBlockOff = kMiscOff + 16;  // of each stage: limit0 and tokens of its query block
    static constexpr int kQueueOff = kBlockOff + (8 * kStages + 15) / 16 * 16;
    static constexpr int kLostOff = kQueueOff + kItemQ * int(sizeof(QWork));  // kLostWords
    static constexpr int kSmemBytes = kLostOff + 4 * packed::kLostWords + 1024;
    static_assert(kQueueOff % 16 == 0, "queue entries are 16-byte aligned");
    static constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 256 + D;
    static_assert(kStageBytes % 1024 == 0, "stages keep the 1024-byte swizzle alignment");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
    static_assert(kColDK + D <= kTmemCols, "TMEM budget");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
packed_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                   const BwdParams p) {
    using C = DkvCfg<D>;
    constexpr int NS = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const uint32_t bar0 = base + C::kBarOff;
    auto st_full = [&](int r) { return bar0 + 8u * r; };
    auto st_empty = [&](int r) { return bar0 + 8u * (NS + r); };
    const uint32_t xb = bar0 + 8u * (2 * NS);
    const uint32_t kv_full = xb, kv_empty = xb + 8, s_full = xb + 16, dp_full = xb + 24, p_full = xb + 32,
                   ds_full = xb + 40, dkv_full = xb + 48, drain = xb + 56;
    const uint32_t item_full0 = xb + 64, item_empty0 = xb + 64 + 8 * kItemQ;
    auto stage_off = [&](int r) { return C::kStageOff + r * C::kStageBytes; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    volatile uint32_t* lost = reinterpret_cast<volatile uint32_t*>(smem + C::kLostOff);
    int2* blocks = reinterpret_cast<int2*>(smem + C::kBlockOff);
    KWork* item_q = reinterpret_cast<KWork*>(smem + C::kQueueOff);
    const int rows_used = (128 / p.group) * p.group;  // rows of a query block's box

    if (threadIdx.x == 0) {
        for (int r = 0; r < NS; ++r) {
            ptx::mbar_init(st_full(r), 1);
            ptx::mbar_init(st_empty(r), 1);
        }
        ptx::mbar_init(kv_full, 1);
        ptx::mbar_init(kv_empty, 1);
        ptx::mbar_init(s_full, 1);
        ptx::mbar_init(dp_full, 1);
        ptx::mbar_init(p_full, kEwWarps);
        ptx::mbar_init(ds_full, kEwWarps);
        ptx::mbar_init(dkv_full, 1);
        ptx::mbar_init(drain, 1);
        for (int q = 0; q < kItemQ; ++q) {
            ptx::mbar_init(item_full0 + 8u * q, 1);
            ptx::mbar_init(item_empty0 + 8u * q, kItemConsumers);
        }
        *abort_flag = 0;
        for (int i = 0; i < packed::kLostWords; ++i) lost[i] = 0;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == kLoadWarp && lane == 0) {
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
        ptx::prefetch_tensormap(&tm_do);
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
        ptx::tmem_relinquish();
    }
    // Rows that no box ever writes (128 is no multiple of the group): zeros for good.
    if (warp < kEwWarps && rows_used < 128)
        for (int r = 0; r < NS; ++r) {
            zero_rows<D>(smem + stage_off(r) + C::kStQ, rows_used, threadIdx.x);
            zero_rows<D>(smem + stage_off(r) + C::kStDO, rows_used, threadIdx.x);
        }
    ops::grid_wait();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int32_t K = p.kv_heads;

    if (warp == kLoadWarp) {
        if (lane == 0) {
            // ------------------------------------------------------------ load
            const int32_t n_items = p.v.lists->w_k * K;
            uint32_t sit = 0, kvc = 0;
            bool ok = !p.inject || wait_bw(drain, 0, abort_flag, p);  // (arrived at on the way out only)
            for (uint32_t kq = 0; ok; ++kq) {
                KWork kb;
                if (!put_item(kq, kb, p.v.kwalks, &p.v.lists->next_k, n_items, K, item_full0, item_empty0, item_q, abort_flag, p))
                    break;
                const int32_t hk = kb.hk;
                if (kb.n == 0) continue;  // no query sees these keys: the elementwise warps write their zeros
                if (!wait_bw(kv_empty, (kvc & 1u) ^ 1u, abort_flag, p)) break;
                ptx::mbar_arrive_expect_tx(kv_full, 2 * C::kBlk);
                load_block<D>(base + C::kKOff, &tm_k, kv_full, hk, kb.key0);
                load_block<D>(base + C::kVOff, &tm_v, kv_full, hk, kb.key0);
                ++kvc;
                QBlock next = p.v.qblocks[kb.q0];  // (fetched a step ahead, while the stage is waited for)
                for (int32_t j = 0; j < kb.n; ++j) {
                    const QBlock qb = next;
                    if (j + 1 < kb.n) next = p.v.qblocks[kb.q0 + j + 1];
                    const int r = int(sit % NS);
                    if (sit >= uint32_t(NS) && !wait_bw(st_empty(r), ((sit / NS) - 1) & 1u, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    const int32_t tok = qb.tok0;
                    blocks[r] = make_int2(qb.limit0, qb.ntok);
                    const int64_t row = (int64_t(kb.q0 + j) * K + hk) * 128;
                    const uint32_t st = base + stage_off(r);
                    ptx::mbar_arrive_expect_tx(st_full(r), 2 * (D / 64) * p.q_box_bytes + 1024);
                    load_block<D>(st + C::kStQ, &tm_q, st_full(r), hk * p.group, tok);
                    load_block<D>(st + C::kStDO, &tm_do, st_full(r), hk * p.group, tok);
                    ptx::bulk_load(st + C::kStL, p.neg_l + row, 512, st_full(r));
                    ptx::bulk_load(st + C::kStD, p.neg_d + row, 512, st_full(r));
                    ++sit;
                }
            }
            for (uint32_t it = sit > uint32_t(NS) ? sit - NS : 0u; it < sit; ++it)
                drain_bar(st_full(int(it % NS)), (it / NS) & 1u, p.timeout_ns);
            if (kvc > 0) drain_bar(kv_full, (kvc - 1) & 1u, p.timeout_ns);
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            // ------------------------------------------------------------- MMA
            constexpr uint32_t idesc_s = ptx::idesc_bf16(128, 128, false);
            constexpr uint32_t idesc_acc = ptx::idesc_bf16(128, D, true);
            const uint32_t kaddr = base + C::kKOff, vaddr = base + C::kVOff;
            uint32_t gs = 0, kvc = 0;
            bool ok = true;
            for (uint32_t kq = 0; ok; ++kq) {
                KWork kb;
                if (!get_item(kq, item_full0, item_q, abort_flag, p, kb)) break;
                ptx::mbar_arrive(item_empty0 + 8u * (kq % kItemQ));
                if (kb.n < 0) break;
                const int32_t n = kb.n;
                // No commit without an arrival of every elementwise warp before it: dkv_full is waited for by
                // parity, and several such items in a row would run phases ahead of a warp that still stores.
                if (n == 0) continue;
                if (!wait_bw(kv_full, kvc & 1u, abort_flag, p)) break;
                ++kvc;
                ptx::tc_fence_after();
                // S^T_j = K Q_j^T (waits for stage j)
                auto issue_s = [&](int32_t j) -> bool {
                    const uint32_t it = gs + uint32_t(j);
                    if (!wait_bw(st_full(int(it % NS)), (it / NS) & 1u, abort_flag, p)) return false;
                    ptx::tc_fence_after();
                    const uint32_t qaddr = base + stage_off(int(it % NS)) + C::kStQ;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t coff = (kk >> 2) * kBoxBytes + (kk & 3) * 32;
                        ptx::mma_ss(tmem + C::kColS, ptx::desc_k_sw128(kaddr + coff), ptx::desc_k_sw128(qaddr + coff),
                                    idesc_s, kk > 0 ? 1u : 0u);
                    }
                    ptx::mma_commit(s_full);
                    return true;
                };
                // dP^T_j = V dO_j^T (stage j already waited for by issue_s)
                auto issue_dp = [&](int32_t j) {
                    const uint32_t it = gs + uint32_t(j);
                    const uint32_t doaddr = base + stage_off(int(it % NS)) + C::kStDO;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t coff = (kk >> 2) * kBoxBytes + (kk & 3) * 32;
                        ptx::mma_ss(tmem + C::kColDP, ptx::desc_k_sw128(vaddr + coff), ptx::desc_k_sw128(doaddr + coff),
                                    idesc_s, kk > 0 ? 1u : 0u);
                    }
                    ptx::mma_commit(dp_full);
                };
                ok = issue_s(0);
                if (ok) issue_dp(0);
                for (int32_t j = 0; ok && j < n; ++j) {
                    const uint32_t it = gs + uint32_t(j);
                    const uint32_t st = base + stage_off(int(it % NS));
                    if (!wait_bw(p_full, it & 1u, abort_flag, p)) { ok = false; break; }
                    ptx::tc_fence_after();
                    // dV += P^T_j dO_j
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        ptx::mma_ts(tmem + C::kColDV, tmem + C::kColS + a_col(kk),
                                    ptx::desc_mn_sw128(st + C::kStDO + kk * 16 * 128, kBoxBytes), idesc_acc,
                                    (j > 0 || kk > 0) ? 1u : 0u);
                    // in issue order after dV_j, which reads the P^T this S^T overwrites
                    if (j + 1 < n && !issue_s(j + 1)) { ok = false; break; }
                    if (!wait_bw(ds_full, it & 1u, abort_flag, p)) { ok = false; break; }
                    ptx::tc_fence_after();
                    // dK += dS^T_j Q_j
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        ptx::mma_ts(tmem + C::kColDK, tmem + C::kColDP + a_col(kk),
                                    ptx::desc_mn_sw128(st + C::kStQ + kk * 16 * 128, kBoxBytes), idesc_acc,
                                    (j > 0 || kk > 0) ? 1u : 0u);
                    ptx::mma_commit(st_empty(int(it % NS)));
                    // after dK_j, which reads the dS^T this dP^T overwrites
                    if (j + 1 < n) issue_dp(j + 1);
                }
                if (!ok) break;
                ptx::mma_commit(dkv_full);
                ptx::mma_commit(kv_empty);
                gs += uint32_t(n);
            }
            ptx::mma_commit(drain);
            drain_bar(drain, 0, p.timeout_ns);
        }
    } else {
        // ------------------------------------------------------- elementwise
        const int h = warp >> 2;  // which 32 query columns
        // Is this part's last column a row that no box fills?  Those are zeros, and so are their products with a
        // key or value, or NaN where that is not finite: the last column says so for all of them.
        const bool gap = rows_used < 32 * h + 32;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = uint32_t((warp & 3) * 32) << 16;
        const uint64_t c2 = ptx::f2(p.scale_log2, p.scale_log2);
        uint32_t gs = 0, kvc = 0;
        bool ok = true;
        for (uint32_t kq = 0; ok; ++kq) {
            KWork kb;
            if (!__all_sync(~0u, get_item(kq, item_full0, item_q, abort_flag, p, kb))) break;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(item_empty0 + 8u * (kq % kItemQ));
            if (kb.n < 0) break;
            const int32_t hk = kb.hk, n = kb.n;
            // 32 columns of dV or dK for each warpgroup, or (d = 64: four 32s in all) of one of them
            const int col = D == 128 ? 32 * h : 32 * (h & 1);
            const bool with_dv = D == 128 || h < 2, with_dk = D == 128 || h >= 2;
            auto row_of = [&](const Rows& x) { return x.p + int64_t(kb.key0 + row) * x.ts + hk * x.hs + col; };
            if (n == 0) {  // zeros, and nothing to wait for (such walks are whole)
                if (with_dv && row < kb.nkeys) zero_cols(row_of(p.out_b));
                if (with_dk && row < kb.nkeys) zero_cols(row_of(p.out_a));
                continue;
            }
            for (int32_t j = 0; j < n; ++j) {
                const uint32_t step = gs + uint32_t(j);
                const int r = int(step % NS);
                // the stage's per-column constants (TMA-written) and the scores
                if (!__all_sync(~0u, wait_bw(st_full(r), (step / NS) & 1u, abort_flag, p) &&
                                         wait_bw(s_full, step & 1u, abort_flag, p))) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                uint8_t* st = smem + stage_off(r);
                const int32_t limit0 = blocks[r].x, rows = blocks[r].y * p.group;
                const bool ragged = rows < rows_used;
                // query rows [from, to) of this part see this thread's key
                const int from = (p.causal ? p.group * max(0, kb.pos + row - limit0 + 1) : 0) - 32 * h, to = rows - 32 * h;
                const bool diagonal = p.causal && kb.pos + 127 >= limit0, masked = ragged || diagonal;
                // rows that do not see every key of the block
                const int partly = diagonal ? min(rows, p.group * (kb.pos + 128 - limit0)) : 0;
                // A Q or dO row that is not finite has an LSE or a D that is not (its products with anything are not;
                // a row that sees no key has LSE = -inf as well), so those two say whether to look.
                bool suspect = false;
                if (partly > 0) {
                    const float4 l = reinterpret_cast<const float4*>(st + C::kStL)[lane];
                    const float4 dd = reinterpret_cast<const float4*>(st + C::kStD)[lane];
                    const float z[4] = {l.x - l.x + (dd.x - dd.x), l.y - l.y + (dd.y - dd.y), l.z - l.z + (dd.z - dd.z),
                                        l.w - l.w + (dd.w - dd.w)};  // 0, or NaN
#pragma unroll
                    for (int i = 0; i < 4; ++i) suspect |= z[i] != 0.0f && 4 * lane + i < partly;
                    suspect = __any_sync(~0u, suspect);
                }
                if (suspect) {
                    // dP must have read them first
                    if (!__all_sync(~0u, wait_bw(dp_full, step & 1u, abort_flag, p))) {
                        ok = false;
                        break;
                    }
                    if (packed::scrub_rows<D / 64>(st + C::kStDO, kBoxBytes, 0, partly, threadIdx.x, kEwThreads))
                        lost[kq % packed::kLostWords] = kq + 1;
                    ptx::fence_proxy_async_smem();
                }
                if (ragged) zero_rows<D>(st + C::kStDO, rows, threadIdx.x);
                // per-column constants, 16-byte broadcast loads
                const float4* cl = reinterpret_cast<const float4*>(st + C::kStL) + 8 * h;
                const float4* cd = reinterpret_cast<const float4*>(st + C::kStD) + 8 * h;
                const uint32_t ts = tmem + lane_addr + C::kColS + 32u * h;
                float pr[32];
                uint32_t pk[16];
                {
                    uint32_t sr[32];
                    ptx::tmem_ld32(ts, sr);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 l = cl[i];
                        float x0, x1, x2, x3;
                        ptx::f2_split(ptx::f2_fma(ptx::f2(__uint_as_float(sr[4 * i]), __uint_as_float(sr[4 * i + 1])),
                                                  c2, ptx::f2(l.x, l.y)),
                                      x0, x1);
                        ptx::f2_split(ptx::f2_fma(ptx::f2(__uint_as_float(sr[4 * i + 2]), __uint_as_float(sr[4 * i + 3])),
                                                  c2, ptx::f2(l.z, l.w)),
                                      x2, x3);
                        pr[4 * i] = ptx::ex2(x0);
                        pr[4 * i + 1] = ptx::ex2(x1);
                        pr[4 * i + 2] = ptx::ex2(x2);
                        pr[4 * i + 3] = ptx::ex2(x3);
                    }
                }
                if (masked || (gap && __any_sync(~0u, pr[31] != pr[31])))
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i < from || i >= to) pr[i] = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) pk[i] = ptx::pack_bf16x2(pr[2 * i], pr[2 * i + 1]);
                ops::tmem_st16(ts, pk);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(p_full);
                if (suspect) {
                    if (packed::scrub_rows<D / 64>(st + C::kStQ, kBoxBytes, 0, partly, threadIdx.x, kEwThreads))
                        lost[kq % packed::kLostWords] = kq + 1;
                    ptx::fence_proxy_async_smem();
                }
                if (ragged) zero_rows<D>(st + C::kStQ, rows, threadIdx.x);
                if (!__all_sync(~0u, wait_bw(dp_full, step & 1u, abort_flag, p))) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t tdp = tmem + lane_addr + C::kColDP + 32u * h;
                {
                    uint32_t dr[32];
                    ptx::tmem_ld32(tdp, dr);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 dd = cd[i];
                        float t0, t1, t2, t3;
                        ptx::f2_split(ptx::f2_mul(ptx::f2(pr[4 * i], pr[4 * i + 1]),
                                                  ptx::f2_add(ptx::f2(__uint_as_float(dr[4 * i]),
                                                                      __uint_as_float(dr[4 * i + 1])),
                                                              ptx::f2(dd.x, dd.y))),
                                      t0, t1);
                        ptx::f2_split(ptx::f2_mul(ptx::f2(pr[4 * i + 2], pr[4 * i + 3]),
                                                  ptx::f2_add(ptx::f2(__uint_as_float(dr[4 * i + 2]),
                                                                      __uint_as_float(dr[4 * i + 3])),
                                                              ptx::f2(dd.z, dd.w))),
                                      t2, t3);
                        pk[2 * i] = ptx::pack_bf16x2(t0, t1);
                        pk[2 * i + 1] = ptx::pack_bf16x2(t2, t3);
                    }
                    if (masked || (gap && __any_sync(~0u, (pk[15] & 0x7f800000u) == 0x7f800000u)))  // (selected last: dP and D of a row may be anything)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            if (2 * i < from || 2 * i >= to) pk[i] &= 0xffff0000u;
                            if (2 * i + 1 < from || 2 * i + 1 >= to) pk[i] &= 0xffffu;
                        }
                }
                ops::tmem_st16(tdp, pk);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ds_full);
            }
            if (!ok) break;
            if (!__all_sync(~0u, wait_bw(dkv_full, kvc & 1u, abort_flag, p))) break;
            ++kvc;
            ptx::tc_fence_after();
            const bool real = row < kb.nkeys;
            // Tokens whose rows may have lost something and see this thread's key: a token that sees `limit`
            // keys is the (limit - limit0)-th from the walk's first.
            const bool fix = lost[kq % packed::kLostWords] == kq + 1;
            auto put_back = [&](const Rows& x, uint32_t (&r)[32]) {
                if (!fix) return;
                const QBlock b0 = p.v.qblocks[kb.q0], b1 = p.v.qblocks[kb.q0 + n - 1];
                const int lo = max(kb.pos + row + 1, b0.limit0), hi = min(kb.pos + 127, b1.limit0 + b1.ntok - 1);
                for (int t = lo; t <= hi; ++t)
                    packed::restore(r, x.p + (int64_t(b0.tok0) + t - b0.limit0) * x.ts + hk * p.group * x.hs + col,
                                    x.hs, p.group);
            };
            auto back_q = [&](uint32_t (&r)[32]) { put_back(p.q, r); };
            auto back_do = [&](uint32_t (&r)[32]) { put_back(p.dout, r); };
            const uint32_t t_dk = tmem + lane_addr + C::kColDK + uint32_t(col), t_dv = tmem + lane_addr + C::kColDV + uint32_t(col);
            if (kb.slot >= 0) {
                float4* part = reinterpret_cast<float4*>(p.v.parts + (int64_t(kb.slot) * K + hk) * (2 * 128 * D)) +
                               col / 4 * 128 + row;
                if (with_dk) store_part(t_dk, part, real, back_q);
                if (with_dv) store_part(t_dv, part + 128 * D / 4, real, back_do);
            } else {
                if (with_dv) store_cols(t_dv, 1.0f, row_of(p.out_b), real, false, back_do);
                if (with_dk) store_cols(t_dk, p.scale, row_of(p.out_a), real, false, back_q);
            }
            ptx::tc_fence_before();
            gs += uint32_t(n);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- parts
// Sums of the parts of split blocks, in their order: dQ (kKeys = false), or dK and dV.  16 bytes
// of the result for each thread; blockIdx.y: 256 threads' worth of a block.
template <int D, bool kKeys>
__global__ void __launch_bounds__(256) packed_sum_kernel(const BwdParams p) {
    ops::grid_wait();
    const int K = p.kv_heads;
    const int64_t n = int64_t(kKeys ? p.v.lists->n_k : p.v.lists->n_q) * K;
    for (int64_t w = blockIdx.x; w < n; w += gridDim.x) {
        const int hk = int(w % K);
        int32_t split, slot, rows, row0;
        if (kKeys) {
            const KBlock b = p.v.kblocks[w / K];
            split = b.split;
            slot = b.slot;
            rows = b.nkeys;
            row0 = b.key0;
        } else {
            const QBlock b = p.v.qblocks[w / K];
            split = b.split;
            slot = b.slot;
            rows = b.ntok * p.group;
            row0 = b.tok0;
        }
        if (split < 2) continue;
        constexpr int kPlanes = kKeys ? 2 : 1;
        const int i = blockIdx.y * 256 + threadIdx.x;
        // a warp: eight rows by four pieces, whole lines of the parts and 64 bytes of a result's row
        const int plane = i / (128 * D / 8), row = i / D % 16 * 8 + i % 8, col = i / 8 % (D / 8) * 8;
        if (plane < kPlanes && row < rows) {
            float x[8] = {};
#pragma unroll 4
            for (int k = 0; k < split; ++k) {
                const float4* src = reinterpret_cast<const float4*>(
                    p.v.parts + ((int64_t(slot + k) * K + hk) * kPlanes + plane) * (128 * D)) + col / 4 * 128 + row;
                const float4 a = src[0], b = src[128];
                x[0] += a.x;
                x[1] += a.y;
                x[2] += a.z;
                x[3] += a.w;
                x[4] += b.x;
                x[5] += b.y;
                x[6] += b.z;
                x[7] += b.w;
            }
            const float mul = plane == 0 ? p.scale : 1.0f;
            const Rows& out = plane == 0 ? p.out_a : p.out_b;
            const int64_t tok = row0 + (kKeys ? row : row / p.group);
            const int head = kKeys ? hk : hk * p.group + row % p.group;
            *reinterpret_cast<uint4*>(out.p + tok * out.ts + head * out.hs + col) =
                make_uint4(ptx::pack_bf16x2(x[0] * mul, x[1] * mul), ptx::pack_bf16x2(x[2] * mul, x[3] * mul),
                           ptx::pack_bf16x2(x[4] * mul, x[5] * mul), ptx::pack_bf16x2(x[6] * mul, x[7] * mul));
        }
    }
}

// ---------------------------------------------------------------- no queries, or no keys
// Gradients of sequences whose other side is empty: zeros.
__global__ void packed_zero_dq_kernel(const PackedProblem p, const packed::View v, int head_dim, Rows dq) {
    ops::grid_wait();
    const int parts = head_dim / 8;
    for (int e = blockIdx.x; e < v.lists->n_q; e += gridDim.x) {
        const QBlock q = v.qblocks[e];
        for (int i = threadIdx.x; i < q.ntok * p.heads * parts; i += blockDim.x) {
            const int row = i / parts;
            *reinterpret_cast<uint4*>(dq.p + int64_t(q.tok0 + row / p.heads) * dq.ts + row % p.heads * dq.hs +
                                      i % parts * 8) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}
__global__ void packed_zero_dkdv_kernel(const PackedProblem p, const packed::View v, int head_dim, Rows dk, Rows dv) {
    ops::grid_wait();
    const int parts = head_dim / 8;
    for (int e = blockIdx.x; e < v.lists->n_k; e += gridDim.x) {
        const KBlock k = v.kblocks[e];
        for (int i = threadIdx.x; i < k.nkeys * p.kv_heads * parts; i += blockDim.x) {
            const int row = i / parts, h = row % p.kv_heads;
            const int64_t tok = k.key0 + row / p.kv_heads;
            *reinterpret_cast<uint4*>(dk.p + tok * dk.ts + h * dk.hs + i % parts * 8) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(dv.p + tok * dv.ts + h * dv.hs + i % parts * 8) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

template <int D>
cudaError_t launch_bwd(const PackedProblem& p, const Rows& q, const Rows& k, const Rows& v, const Rows& o,
                       const Rows& dout, const float* lse, const Rows& dq, const Rows& dk, const Rows& dv, char* ws,
                       const packed::Layout& w, const packed::View& view, int sms, cudaStream_t stream) {
    const int tpb = 128 / p.group;
    CUtensorMap mq, mk, mv, md;
    cudaError_t e = packed::rows_map(&mq, q, p.tokens_q, p.heads, D, p.group, tpb);
    if (e == cudaSuccess) e = packed::rows_map(&md, dout, p.tokens_q, p.heads, D, p.group, tpb);
    if (e == cudaSuccess) e = packed::rows_map(&mk, k, p.tokens_k, p.kv_heads, D, 1, 128);
    if (e == cudaSuccess) e = packed::rows_map(&mv, v, p.tokens_k, p.kv_heads, D, 1, 128);
    if (e != cudaSuccess) return e;
    float* neg_l = reinterpret_cast<float*>(ws + w.neg_l);
    float* neg_d = reinterpret_cast<float*>(ws + w.neg_d);
    BwdParams bp{view, p.kv_heads, p.group, p.causal, neg_l, neg_d, dq, dq, p.scale, p.scale * kLog2e,
                 uint32_t(p.group * tpb) * 128u, p.status, p.waits.timeout_ns, p.waits.inject, q, k, dout};
    constexpr int kDq = smem_launch(DqCfg<D>::kSmemBytes), kDkv = smem_launch(DkvCfg<D>::kSmemBytes);
    e = cudaFuncSetAttribute(packed_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDq);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(packed_dkdv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDkv);
    const int64_t nq = w.max_q * p.kv_heads, nk = w.max_k * p.kv_heads;
    const int64_t wq = w.max_wq * p.kv_heads, wk = w.max_wk * p.kv_heads;
    auto grid = [&](int64_t n, int64_t most) { return dim3(unsigned(n < most ? n : most)); };
    if (e == cudaSuccess)
        e = packed::launch(packed_prep_kernel<D>, grid(nq, 4 * sms), 256, 0, stream, true, p, view, o, dout, lse, neg_l, neg_d);
    if (e == cudaSuccess)
        e = packed::launch(packed_dq_kernel<D>, grid(wq, sms), kThreads, kDq, stream, true, mq, mk, mv, md, bp);
    if (e == cudaSuccess && w.split_q)
        e = packed::launch(packed_sum_kernel<D, false>, dim3(unsigned(nq), D / 16), 256, 0, stream, true, bp);
    bp.out_a = dk;
    bp.out_b = dv;
    if (e == cudaSuccess)
        e = packed::launch(packed_dkdv_kernel<D>, grid(wk, sms), kThreads, kDkv, stream, true, mq, mk, mv, md, bp);
    if (e == cudaSuccess && w.split_k)
        e = packed::launch(packed_sum_kernel<D, true>, dim3(unsigned(nk), D / 8), 256, 0, stream, true, bp);
    return e;
}

}  // namespace

cudaError_t launch_packed_backward(const PackedProblem& p, int head_dim, const Rows& q, const Rows& k, const Rows& v,
                                   const Rows& o, const Rows& dout, const float* lse, const Rows& dq, const Rows& dk,
                                   const Rows& dv, void* workspace, cudaStream_t stream) {
    int sms = 0;
    if (cudaError_t e = packed::sm_count(&sms); e != cudaSuccess) return e;
    const packed::Layout w = packed::layout(p, true, head_dim, sms);
    const packed::View view = packed::view(w, workspace);
    packed::Tails tails{};
    tails.r[0] = dq;
    tails.r[1] = dk;
    tails.r[2] = dv;
    tails.heads[0] = p.heads;
    tails.heads[1] = tails.heads[2] = p.kv_heads;
    tails.is_q[0] = 1;
    tails.n = 3;
    const cudaError_t e = packed::launch_lists(p, view, true, head_dim, tails, stream);
    if (e != cudaSuccess || p.batch == 0) return e;
    if (p.tokens_k == 0)
        return packed::launch(packed_zero_dq_kernel, dim3(unsigned(sms)), 256, 0, stream, true, p, view, head_dim, dq);
    if (p.tokens_q == 0)
        return packed::launch(packed_zero_dkdv_kernel, dim3(unsigned(sms)), 256, 0, stream, true, p, view, head_dim, dk, dv);
    if (head_dim == 128)
        return launch_bwd<128>(p, q, k, v, o, dout, lse, dq, dk, dv, static_cast<char*>(workspace), w, view, sms, stream);
    return launch_bwd<64>(p, q, k, v, o, dout, lse, dq, dk, dv, static_cast<char*>(workspace), w, view, sms, stream);
}

}  // namespace sta
