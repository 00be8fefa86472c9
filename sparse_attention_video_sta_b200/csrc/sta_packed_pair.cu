// sta_packed_pair.cu -- the packed forward for short walks: two items at a time on an SM.
//
// The kernel of sta_packed.cu splits each chunk of keys between both softmax warpgroups and
// runs up to three chunks ahead: best where a walk has many chunks.  A walk of one to a few
// chunks is mostly beginning and end -- loads, the first maximum, the last product, the
// stores -- and those follow one another.  Here each softmax warpgroup has an item of its own
// (128 rows, whole chunks of 128 keys), with its own load warp, tcgen05 issuing thread, S, O
// and buffers; nothing orders the two, so one item's beginnings and ends are covered by the
// other's exponentials.  The price is that an item's own steps follow one another, S(i + 1)
// after P(i) V: P lies over S, and TMEM holds two S and two O.
//
//   warps 0-3, 4-7 : softmax of slot 0, 1 (a thread for each row)
//   warps 8, 9     : loads of slot 0, 1
//   warps 10, 11   : S = Q K^T and O += P V of slot 0, 1
//   warps 12-15    : O / l of both slots, whichever is done, to memory, while the softmax goes on
//
// Masks and rows that are not there: as in sta_packed.cu; V rows that no row of the block sees are
// cleared by the softmax warpgroup before it hands over its P.
// Measured: 20736 queries of two videos on 226 and 100 text keys, 24 heads, d = 128: 101-106 us (152 one item
// at a time; 117 with the softmax warps storing O themselves; the tensors alone are 40 us of HBM).  No unit
// is busy for more than a third of the time: an item's steps follow one another (loads, product, maximum,
// exponentials, product), and TMEM holds no third S and O.
// The storing warps turn their 32 rows through shared memory, so that a store instruction
// writes 128 bytes of four rows, not 16 of 32.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sta_ops.cuh"
#include "sta_ops.h"
#include "sta_packed.cuh"
#include "sta_packed_fwd.cuh"
#include "sta_ptx.cuh"
#include "sta_wait.cuh"

namespace sta {
namespace {

using namespace packed_fwd;

constexpr int kThreads = 512;
constexpr int kLoadWarp = 8, kMmaWarp = 10;  // + slot
constexpr int kStoreWarp = 12;
// (20736 queries on text keys: 102 us so; 176 / 64 / 96: 109, 192 / 48 / 80: 119, 192 / 56 / 72: 108.)
constexpr uint32_t kRegsSoftmax = 184, kRegsProducer = 64, kRegsStore = 80;
static_assert(128 * (2 * kRegsSoftmax + kRegsProducer + kRegsStore) <= kThreads * 128, "register split exceeds the launch");
constexpr uint32_t kTmemCols = 512;
constexpr int kConsumers = 1 + 4 + 4;  // of a slot's items: the issuing thread, the softmax and the storing warps
// log2 by which scores may pass the running maximum before O and l are rescaled
constexpr float kRise = 8.0f;

template <int D>
struct PairCfg {
    static constexpr int kColBlocks = D / 64;
    static constexpr int kBlk = 128 * D * 2;
    static constexpr int kStages = D == 128 ? 1 : 2;  // of K and of V, for each slot
    static constexpr int kSlotBytes = kBlk * (1 + 2 * kStages);
    static constexpr int kStageOff = 2 * kSlotBytes;  // 4 KB for each storing warp
    static constexpr int kSumOff = kStageOff + 4 * 4096;  // l of an item's rows: [2 slots][2 items][128] fp32
    static constexpr int kBarOff = kSumOff + 2 * 2 * 512;
    // of each slot: q_full, q_empty, k_full[S], k_empty[S], v_full[S], v_empty[S], s_full, p_full,
    // o_full, o_empty, drain, item_full[Q], item_empty[Q]
    static constexpr int kSlotBars = 2 + 4 * kStages + 5 + 2 * kItemQ;
    static constexpr int kQueueOff = kBarOff + (2 * kSlotBars + 1) / 2 * 16;
    static constexpr int kMiscOff = kQueueOff + 2 * kItemQ * int(sizeof(QWork));  // tmem base slot, abort flag
    static constexpr int kLostOff = kMiscOff + 16;  // of each slot kLostWords
    static constexpr int kSmemBytes = kLostOff + 2 * 4 * packed::kLostWords + 1024;
    static constexpr uint32_t kColO = 256;
    static_assert(kQueueOff % 16 == 0, "queue entries are 16-byte aligned");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
    static_assert(kColO + 2 * D <= int(kTmemCols), "TMEM budget");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
packed_fwd_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const FwdParams p) {
    using C = PairCfg<D>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = warp < 8 ? warp >> 2 : warp & 1;  // (the storing warps serve both)

    const uint32_t bar0 = base + C::kBarOff + uint32_t(slot) * (C::kSlotBars * 8);
    const uint32_t q_full = bar0, q_empty = bar0 + 8;
    auto k_full = [&](int r) { return bar0 + 16 + 8u * r; };
    auto k_empty = [&](int r) { return bar0 + 16 + 8u * (S + r); };
    auto v_full = [&](int r) { return bar0 + 16 + 8u * (2 * S + r); };
    auto v_empty = [&](int r) { return bar0 + 16 + 8u * (3 * S + r); };
    const uint32_t xb = bar0 + 16 + 32 * S;
    const uint32_t s_full = xb, p_full = xb + 8, o_full = xb + 16, o_empty = xb + 24, drain = xb + 32;
    auto item_full = [&](int q) { return xb + 40 + 8u * q; };
    auto item_empty = [&](int q) { return xb + 40 + 8u * (kItemQ + q); };
    QWork* item_q = reinterpret_cast<QWork*>(smem + C::kQueueOff) + slot * kItemQ;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile uint32_t* lost = reinterpret_cast<volatile uint32_t*>(smem + C::kLostOff) + slot * packed::kLostWords;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    const uint32_t q_at = base + uint32_t(slot) * C::kSlotBytes, k_at = q_at + C::kBlk, v_at = k_at + S * C::kBlk;
    auto wait_bar = [&](uint32_t bar, uint32_t parity) {
        return wait_bar_limited(bar, parity, abort_flag, p.status, p.timeout_ns);
    };
    auto take_item = [&](uint32_t k, QWork& w) -> bool {
        if (!wait_bar(item_full(int(k % kItemQ)), (k / kItemQ) & 1u)) return false;
        w = item_q[k % kItemQ];
        return true;
    };

    if (threadIdx.x == 256 || threadIdx.x == 288) {  // the load warps' first lanes, each for its slot
        ptx::mbar_init(q_full, 1);
        ptx::mbar_init(q_empty, 1);
        for (int r = 0; r < S; ++r) {
            ptx::mbar_init(k_full(r), 1);
            ptx::mbar_init(k_empty(r), 1);
            ptx::mbar_init(v_full(r), 1);
            ptx::mbar_init(v_empty(r), 1);
        }
        ptx::mbar_init(s_full, 1);
        ptx::mbar_init(p_full, 4);
        ptx::mbar_init(o_full, 1);
        ptx::mbar_init(o_empty, 4);
        ptx::mbar_init(drain, 1);
        for (int q = 0; q < kItemQ; ++q) {
            ptx::mbar_init(item_full(q), 1);
            ptx::mbar_init(item_empty(q), kConsumers);
        }
        if (slot == 0) *abort_flag = 0;
        for (int i = 0; i < packed::kLostWords; ++i) lost[i] = 0;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
        ptx::tmem_relinquish();
    }
    ops::grid_wait();  // the lists
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem + uint32_t(slot) * 128u, tO = tmem + C::kColO + uint32_t(slot) * D;
    const int32_t K = p.kv_heads;
    // this slot among all: every CTA's first, then every CTA's second
    const int32_t id = slot * int32_t(gridDim.x) + int32_t(blockIdx.x), ids = int32_t(gridDim.x) * 2;

    if (warp >= kLoadWarp && warp < kLoadWarp + 2) {
        ptx::regs_dec<kRegsProducer>();
        if (p.self) self_items(p.prob, item_q, id, ids);
        if (lane == 0) {
            // ------------------------------------------------------------ load
            const int32_t n_items = p.self ? 0 : p.v.lists->w_q * K;
            auto fetch = [&](int32_t u) {
                QWork w{};
                w.n = -1;
                if (u < n_items) {
                    w = p.v.qwalks[u / K];
                    w.hk = u % K;
                }
                return w;
            };
            // the first item is the slot's own number; the counter's answer for item k + 2 and the
            // walk of item k + 1 are on their way while item k's copies are issued, if items are many
            const bool early = !p.self && n_items >= 8 * ids;
            auto next = [&] { return ids + atomicAdd(&p.v.lists->next_q, 1); };
            int32_t u2 = early ? next() : 0;
            QWork w1 = p.self ? item_q[0] : fetch(id);
            uint32_t ki = 0, vi = 0, qi = 0;
            bool ok = !p.prob.waits.inject || wait_bar(drain, 0);  // (arrived at on the way out only)
            for (uint32_t k = 0; ok; ++k) {
                const int qe = int(k % kItemQ);
                if (k > 0 && p.self)
                    w1 = item_q[qe];  // (the last entry is an end)
                else if (k > 0 && !early)
                    w1 = fetch(next());
                const QWork q = w1;
                if (k >= uint32_t(kItemQ) && !wait_bar(item_empty(qe), ((k / kItemQ) - 1) & 1u)) break;
                if (!p.self) item_q[qe] = q;
                ptx::mbar_arrive(item_full(qe));
                if (q.n < 0) break;
                if (early) {
                    w1 = fetch(u2);
                    if (u2 < n_items) u2 = next();
                }
                const int32_t row0 = q.key0 + q.c0 * 128;
                if (!wait_bar(q_empty, (qi & 1u) ^ 1u)) break;
                ptx::mbar_arrive_expect_tx(q_full, C::kColBlocks * p.q_box_bytes);
#pragma unroll
                for (int cb = 0; cb < C::kColBlocks; ++cb)
                    ops::tma_load_3d(q_at + cb * kBoxBytes, &tm_q, q_full, cb * 64, q.hk * p.group, q.tok0);
                ++qi;
                auto load = [&](const CUtensorMap* m, uint32_t full, uint32_t empty, uint32_t at, uint32_t it, int32_t row) {
                    if (it >= uint32_t(S) && !wait_bar(empty, ((it / S) - 1) & 1u)) return false;
                    ptx::mbar_arrive_expect_tx(full, C::kBlk);
#pragma unroll
                    for (int cb = 0; cb < C::kColBlocks; ++cb)
                        ops::tma_load_3d(at + (it % S) * C::kBlk + cb * kBoxBytes, m, full, cb * 64, q.hk, row);
                    return true;
                };
                for (int32_t i = 0; i < q.n; ++i) {
                    ok = load(&tm_k, k_full(int(ki % S)), k_empty(int(ki % S)), k_at, ki, row0 + i * 128);
                    if (!ok) break;
                    ++ki;
                    ok = load(&tm_v, v_full(int(vi % S)), v_empty(int(vi % S)), v_at, vi, row0 + i * 128);
                    if (!ok) break;
                    ++vi;
                }
            }
            // Drain the copies that may still be in flight (after an abort).
            for (uint32_t it = ki > uint32_t(S) ? ki - S : 0u; it < ki; ++it)
                drain_bar(k_full(int(it % S)), (it / S) & 1u, p.timeout_ns);
            for (uint32_t it = vi > uint32_t(S) ? vi - S : 0u; it < vi; ++it)
                drain_bar(v_full(int(it % S)), (it / S) & 1u, p.timeout_ns);
            if (qi > 0) drain_bar(q_full, (qi - 1) & 1u, p.timeout_ns);
        }
        __syncwarp();
        if (p.self && p.prob.clear_tail && slot == 0) self_clear(p.prob, D, p.o, p.lse);
    } else if (warp >= kStoreWarp) {
        ptx::regs_dec<kRegsStore>();
        // ------------------------------------------------------------ O / l -> bf16
        const int row = threadIdx.x & 127;
        uint8_t* stage = smem + C::kStageOff + (warp - kStoreWarp) * 4096;
        const int r_tok = row / p.group, r_head = row - r_tok * p.group;
        uint32_t done[2] = {0u, 0u};  // items of each slot
        bool live[2] = {true, true};
        int32_t steps[2] = {0, 0};  // chunks of the items under way
        uint64_t since = 0;
        uint32_t idle = 0;
        while (live[0] || live[1]) {
            bool moved = false;
#pragma unroll 1
            for (int s = 0; s < 2; ++s) {
                if (!live[s]) continue;
                const uint32_t kq = done[s], b = base + C::kBarOff + uint32_t(s) * (C::kSlotBars * 8) + 16 + 32 * S;
                const uint32_t o_full_s = b + 16, o_empty_s = b + 24, full = b + 40 + 8u * (kq % kItemQ),
                               empty = b + 40 + 8u * (kItemQ + kq % kItemQ);
                if (!__all_sync(~0u, ptx::mbar_test_wait(full, (kq / kItemQ) & 1u))) continue;
                const QWork* item = reinterpret_cast<const QWork*>(smem + C::kQueueOff) + s * kItemQ + kq % kItemQ;
                steps[s] = item->n;
                if (steps[s] < 0) {
                    live[s] = false;
                    steps[s] = 0;
                    continue;
                }
                if (!__all_sync(~0u, ptx::mbar_test_wait(o_full_s, kq & 1u))) continue;
                const QWork q = *item;
                __syncwarp();
                moved = true;
                steps[s] = 0;
                ++done[s];
                if (lane == 0) ptx::mbar_arrive(empty);
                ptx::tc_fence_after();
                const uint32_t mO = tmem + C::kColO + uint32_t(s) * D + (uint32_t((warp & 3) * 32) << 16);
                const bool real = r_tok < q.ntok;
                const int limit = real ? min(q.nkeys, q.limit0 + (p.causal ? r_tok : 0)) : 0;
                const float l = reinterpret_cast<const float*>(smem + C::kSumOff)[(s * 2 + int(kq & 1u)) * 128 + row];
                const bool none = l == 0.0f;  // no visible key: O = 0, whatever TMEM holds
                const int32_t head = q.hk * p.group + r_head;
                const int64_t tok = q.tok0 + r_tok;
                const volatile uint32_t* lost_s =
                    reinterpret_cast<const volatile uint32_t*>(smem + C::kLostOff) + s * packed::kLostWords;
                const bool fix = real && lost_s[kq % packed::kLostWords] == kq + 1;
                int lo;
                const int seen = lost_seen(q, limit, lo);
                const __nv_bfloat16* seen_v = p.vals.p + (q.key0 + int64_t(lo)) * p.vals.ts + q.hk * p.vals.hs;
                if (q.slot >= 0) {
                    float* part = p.v.parts + (int64_t(q.slot) * K + q.hk) * (128 * (D + 2));
#pragma unroll 1
                    for (int cb = 0; cb < D / 32; ++cb) {
                        uint32_t orr[32];
                        ptx::tmem_ld32(mO + cb * 32, orr);
                        if (fix) packed::restore(orr, seen_v + cb * 32, p.vals.ts, seen);
                        float4* d4 = reinterpret_cast<float4*>(part) + cb * 8 * 128 + row;
                        if (real)
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                d4[j * 128] = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                             : make_float4(__uint_as_float(orr[4 * j]), __uint_as_float(orr[4 * j + 1]),
                                                           __uint_as_float(orr[4 * j + 2]), __uint_as_float(orr[4 * j + 3]));
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(o_empty_s);
                } else {
                    const float inv = none ? 0.0f : 1.0f / l;
                    const uint64_t inv2 = ptx::f2(inv, inv);
                    const int64_t out = real ? tok * p.o.ts + head * p.o.hs : -1;  // element offset of this thread's row
#pragma unroll 1
                    for (int cb = 0; cb < D / 64; ++cb) {  // 64 columns (128 bytes) of the warp's 32 rows at a time
#pragma unroll
                        for (int hc = 0; hc < 2; ++hc) {
                            uint32_t orr[32];
                            ptx::tmem_ld32(mO + cb * 64 + hc * 32, orr);
                            if (fix) packed::restore(orr, seen_v + cb * 64 + hc * 32, p.vals.ts, seen);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t pk[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    float o0, o1;
                                    ptx::f2_split(ptx::f2_mul(ptx::f2(__uint_as_float(orr[8 * j + 2 * e]),
                                                                      __uint_as_float(orr[8 * j + 2 * e + 1])), inv2),
                                                  o0, o1);
                                    pk[e] = none ? 0u : ptx::pack_bf16x2(o0, o1);
                                }
                                *reinterpret_cast<uint4*>(stage + lane * 128 + (((hc * 4 + j) ^ (lane & 7)) << 4)) =
                                    make_uint4(pk[0], pk[1], pk[2], pk[3]);
                            }
                        }
                        if (cb == D / 64 - 1) {  // O is read
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(o_empty_s);
                        }
                        __syncwarp();
#pragma unroll
                        for (int it = 0; it < 8; ++it) {
                            const int r = it * 4 + (lane >> 3), j = lane & 7;
                            const int64_t at = __shfl_sync(~0u, out, r);
                            const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((j ^ (r & 7)) << 4));
                            if (at >= 0) *reinterpret_cast<uint4*>(p.o.p + at + cb * 64 + j * 8) = v;
                        }
                        __syncwarp();
                    }
                }
            }
            // bounded, as every wait; an item may take its chunks' time (some 2 us each)
            if (moved) {
                idle = 0;
            } else {
                if (__any_sync(~0u, *abort_flag != 0)) break;
                if (idle++ == 0) since = ptx::globaltimer_ns();
                if (idle % 64 == 0 && __any_sync(~0u, ptx::globaltimer_ns() - since >
                                                      p.timeout_ns + uint64_t(int64_t(steps[0]) + steps[1]) * 20000u)) {
                    *abort_flag = 1;
                    if (lane == 0) atomicOr(p.status, kDevTimeout);
                    break;
                }
            }
        }
    } else if (warp >= kMmaWarp) {
        ptx::regs_dec<kRegsProducer>();
        if (lane == 0) {
            // ------------------------------------------------------------- MMA
            // One thread issues both products of its slot, so they run in the order of issue:
            // S(i + 1) over the P that O += P(i) V has read; s_full(i + 1) also says that
            // product is done.
            constexpr uint32_t idesc_qk = ptx::idesc_bf16(128, 128, false);
            constexpr uint32_t idesc_pv = ptx::idesc_bf16(128, D, true);
            uint32_t g = 0;
            bool ok = true;
            for (uint32_t kq = 0; ok; ++kq) {
                QWork q;
                if (!take_item(kq, q)) break;
                ptx::mbar_arrive(item_empty(int(kq % kItemQ)));
                if (q.n < 0) break;
                if (!wait_bar(q_full, kq & 1u)) break;
                for (int32_t i = 0; i < q.n; ++i, ++g) {
                    const int r = int(g % S);
                    if (!wait_bar(k_full(r), (g / S) & 1u)) { ok = false; break; }
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t coff = (kk >> 2) * kBoxBytes + (kk & 3) * 32;
                        ptx::mma_ss(tS, ptx::desc_k_sw128(q_at + coff), ptx::desc_k_sw128(k_at + r * C::kBlk + coff), idesc_qk,
                                    kk > 0 ? 1u : 0u);
                    }
                    ptx::mma_commit(s_full);
                    ptx::mma_commit(k_empty(r));
                    if (i == q.n - 1) ptx::mma_commit(q_empty);
                    if (!wait_bar(v_full(r), (g / S) & 1u)) { ok = false; break; }
                    if (i == 0 && !wait_bar(o_empty, (kq & 1u) ^ 1u)) { ok = false; break; }
                    if (!wait_bar(p_full, g & 1u)) { ok = false; break; }
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        ptx::mma_ts(tO, tS + kk * 8, ptx::desc_mn_sw128(v_at + r * C::kBlk + kk * 16 * 128, kBoxBytes),
                                    idesc_pv, (i > 0 || kk > 0) ? 1u : 0u);
                    ptx::mma_commit(v_empty(r));
                }
                if (!ok) break;
                ptx::mma_commit(o_full);
            }
            ptx::mma_commit(drain);
            drain_bar(drain, 0, p.timeout_ns);
        }
    } else {
        // ------------------------------------------------------------- softmax
        ptx::regs_inc<kRegsSoftmax>();
        const int row = threadIdx.x & 127;
        const uint32_t lane_addr = uint32_t((warp & 3) * 32) << 16;
        const uint32_t mS = tS + lane_addr, mO = tO + lane_addr;
        float* sums = reinterpret_cast<float*>(smem + C::kSumOff) + slot * 256 + row;
        const float c = p.scale_log2;
        const int r_tok = row / p.group, r_head = row - r_tok * p.group;
        uint32_t g = 0;
        bool ok = true;
        for (uint32_t kq = 0; ok; ++kq) {
            QWork q;
            q.n = -1;
            if (!__all_sync(~0u, take_item(kq, q))) break;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(item_empty(int(kq % kItemQ)));
            if (q.n < 0) break;
            const bool real = r_tok < q.ntok;
            const int limit = real ? min(q.nkeys, q.limit0 + (p.causal ? r_tok : 0)) : INT32_MAX;
            // over the rows that are stored: below `least` nothing is masked, from `most` on everything
            const int least = __reduce_min_sync(~0u, limit), most = __reduce_max_sync(~0u, real ? limit : INT32_MIN);
            float m = 0.0f, l = 0.0f;
            for (int32_t i = 0; i < q.n; ++i, ++g) {
                if (!__all_sync(~0u, wait_bar(s_full, g & 1u))) { ok = false; break; }
                ptx::tc_fence_after();
                uint32_t s0[64], s1[64];
                ptx::tmem_ld64(mS, s0);
                ptx::tmem_ld64(mS + 64, s1);
                const int key = (q.c0 + i) * 128;
                // 32 keys at a time: masked where some row's limit falls in them, left out where every row's has passed
                const bool cut = key + 128 > least;
                float mx;
                if (!cut) {
                    mx = fmaxf(row_max64(s0), row_max64(s1));
                } else {
                    if (key + 32 > least) mask_from32<0>(s0, limit - key);
                    if (key + 64 > least) mask_from32<32>(s0, limit - key - 32);
                    if (key + 96 > least) mask_from32<0>(s1, limit - key - 64);
                    if (key + 128 > least) mask_from32<32>(s1, limit - key - 96);
                    mx = row_max32<0>(s0);
                    if (key + 32 < most) mx = fmaxf(mx, row_max32<32>(s0));
                    if (key + 64 < most) mx = fmaxf(mx, row_max32<0>(s1));
                    if (key + 96 < most) mx = fmaxf(mx, row_max32<32>(s1));
                }
                float alpha = 1.0f;
                if (i == 0) {
                    m = mx == -INFINITY ? p.nothing_yet : mx;  // (no key, or scores of -inf alone)
                } else if (real && (mx - m) * c > kRise) {
                    alpha = ptx::ex2((m - mx) * c);
                    m = mx;
                }
                if (i > 0 && __any_sync(~0u, alpha != 1.0f)) {  // O holds P(.. i - 1) V: s_full has said so
                    l *= alpha;
                    const uint64_t alpha2 = ptx::f2(alpha, alpha);
#pragma unroll 1
                    for (int cb = 0; cb < D / 32; ++cb) {
                        uint32_t orr[32];
                        ptx::tmem_ld32(mO + cb * 32, orr);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float o0, o1;
                            ptx::f2_split(ptx::f2_mul(ptx::f2(__uint_as_float(orr[2 * j]), __uint_as_float(orr[2 * j + 1])),
                                                      alpha2),
                                          o0, o1);
                            orr[2 * j] = __float_as_uint(o0);
                            orr[2 * j + 1] = __float_as_uint(o1);
                        }
                        ptx::tmem_st32(mO + cb * 32, orr);
                    }
                }
                uint32_t pk[32];
                if (!cut) {
                    l += softmax_exp64(s0, c, m, pk);
                    ptx::tmem_st32(mS, pk);
                    l += softmax_exp64(s1, c, m, pk);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) pk[j] = 0u;
                    l += softmax_exp32<0>(s0, c, m, pk);
                    if (key + 32 < most) l += softmax_exp32<32>(s0, c, m, pk);
                    ptx::tmem_st32(mS, pk);
#pragma unroll
                    for (int j = 0; j < 32; ++j) pk[j] = 0u;
                    if (key + 64 < most) l += softmax_exp32<0>(s1, c, m, pk);
                    if (key + 96 < most) l += softmax_exp32<32>(s1, c, m, pk);
                }
                ptx::tmem_st32(mS + 32, pk);
                if (i >= first_care(q)) {
                    // V rows that no row sees, or not every one (the V in flight or here is this chunk's: the
                    // one before was read by a product that s_full has waited for)
                    const int r = int(g % S);
                    if (!__all_sync(~0u, wait_bar(v_full(r), (g / S) & 1u))) { ok = false; break; }
                    uint8_t* v0 = smem + (v_at - base) + r * C::kBlk;
                    const int dead = dead_from(q, p.causal, key);
                    for (int j = dead * 8 + row; j < 128 * 8; j += 128)
#pragma unroll
                        for (int cb = 0; cb < C::kColBlocks; ++cb)
                            *reinterpret_cast<uint4*>(v0 + cb * kBoxBytes + j * 16) = make_uint4(0u, 0u, 0u, 0u);
                    if (packed::scrub_rows<C::kColBlocks>(v0, kBoxBytes, hidden_from(q, key), dead, row, 128))
                        lost[kq % packed::kLostWords] = kq + 1;
                    ptx::fence_proxy_async_smem();
                }
                // (read after this chunk's product; the item two before has been stored: this one's first product
                // waited for the O of the one before)
                if (i == q.n - 1) sums[(kq & 1u) * 128] = l;
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(p_full);
            }
            if (!ok) break;
            if (real) {
                const bool none = l == 0.0f;
                if (q.slot >= 0)
                    *reinterpret_cast<float2*>(p.v.parts + (int64_t(q.slot) * K + q.hk) * (128 * (D + 2)) + 128 * D + 2 * row) =
                        make_float2(none ? -INFINITY : m * c, l);
                else
                    p.lse[int64_t(q.hk * p.group + r_head) * p.tokens_q + q.tok0 + r_tok] =
                        none ? -INFINITY : m * p.scale + logf(l);
            }
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

template <int D>
cudaError_t launch_pair(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const FwdParams& fp,
                        int64_t items, int sms, cudaStream_t stream) {
    constexpr int kSmem = PairCfg<D>::kSmemBytes;
    cudaError_t e = cudaFuncSetAttribute(packed_fwd_pair_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    return packed::launch(packed_fwd_pair_kernel<D>, dim3(unsigned(items < sms ? items : sms)), kThreads, kSmem, stream, true,
                          mq, mk, mv, fp);
}

}  // namespace

cudaError_t packed_fwd::launch_forward_pair(int head_dim, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                            const FwdParams& fp, int64_t items, int sms, cudaStream_t stream) {
    return head_dim == 128 ? launch_pair<128>(mq, mk, mv, fp, items, sms, stream)
                           : launch_pair<64>(mq, mk, mv, fp, items, sms, stream);
}

}  // namespace sta
