// sta_packed.cu -- attention of packed sequences of different lengths, causal
// or not, with grouped heads: the C entry points and the forward kernel.
//
// Two launches: the work lists from the bounds (sta_packed_lists.cu), and a
// persistent tcgen05 kernel that starts beside it; one launch for small problems, which
// the kernel plans itself; a third where few long walks are split (packed_join_kernel).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "sta_ops.cuh"
#include "sta_ops.h"
#include "sta_packed.cuh"
#include "sta_packed_fwd.cuh"
#include "sta_ptx.cuh"
#include "sta_wait.cuh"

namespace sta {
namespace {

using packed::QBlock;
using packed::QWork;
using namespace packed_fwd;

constexpr int kThreads = 384;  // 3 warpgroups: softmax half A, softmax half B, producers
constexpr int kLoadWarp = 8;
constexpr int kPvWarp = 9;    // PV issuer; also allocates TMEM
constexpr int kSWarp = 10;    // S issuer
constexpr int kTailWarp = 11; // clears V rows behind a sequence's last key
// Registers as in the video kernel: 384 threads launched at 168, the producers
// give theirs to the softmax warpgroups; 128 * (208 + 208 + 88) <= 384 * 168.
constexpr uint32_t kRegsSoftmax = 208;
constexpr uint32_t kRegsProducer = 88;
static_assert(128 * (2 * kRegsSoftmax + kRegsProducer) <= kThreads * 168, "register split exceeds the launch");
constexpr uint32_t kTmemCols = 512;
constexpr int kItemConsumers = 3 + 8;   // the issuing threads, the tail warp and the eight softmax warps
constexpr int kSBufs = 3;               // S buffers in TMEM
// A half-row sum above this takes the slow path (the running maximum is raised).
constexpr float kRescaleRowSum = 65536.0f;


constexpr int kMaxDevices = 64;
__device__ uint32_t g_op_status;  // one word per device: kDevTimeout | kDevBounds
__device__ uint32_t g_op_taken;   // the bit that sta_operator_status took last
std::mutex g_status_mutex, g_taken_mutex;
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per device-side wait
std::atomic<int32_t> g_op_inject_ms{0};
uint32_t* g_status_ptr[kMaxDevices] = {};

// The forward kernel.  One item is one query block (128 rows: tokens x the query
// heads of one key head, sta_packed.cuh) of one key head; the pipeline is the
// video forward's key-split one: every 128-key chunk is split between two
// softmax warpgroups (keys 0-63 and 64-127) that share a running maximum for
// each row and accumulate into one O, S is triple buffered in TMEM.
//
//   warp 8  (load): TMA of the query block (two buffers) and K(0), K(1), K(2), then
//                   V(i), K(i + 3) into the ring
//   warp 9  (PV)  : O += P_A V_A, then O += P_B V_B as each half's P lands in TMEM
//   warp 10 (S)   : S(c) = Q K(c)^T into buffer c % 3, once the PVs of chunk c - 3 are done
//   warp 11 (tail): rows of a V chunk that no row of the block sees (behind the causal diagonal,
//                   or the sequence's end) have P = 0, but 0 x inf is not 0: they are overwritten
//                   with zeros in shared memory, and those that only some rows see lose what is
//                   not finite (scrub_rows)
//   warps 0-7     : softmax halves and the epilogue
//
// Masks: a row sees keys [0, limit).  A chunk wholly below every row's limit
// (warp-uniform test) runs without a mask; in the others scores from the limit
// on become -inf before any arithmetic, so what they were (NaN, inf) is
// forgotten.  Every row that sees a key sees key 0, in half A of chunk 0, so the
// first chunk sets its maximum; a row without keys, or with scores of -inf alone so far,
// gets a stand-in below any other score, and one that stays so ends with l = 0.  Rows past the block's tokens hold whatever the box brought: they
// are never stored, and never start the slow path.
// Bound like the video forward: MUFU exponentials and the tensor pipe nearly level at d = 128
// (16384 causal tokens, 24 / 8 heads: 1.63-1.7 ms, 970-1010 TFLOP/s over the visible pairs; tensor pipe and
// MUFU 56 % each under a profiler's higher clock; what is left is the chunk's round trips and the board's power cap);
// causal blocks lose the masked part of their last chunks.  Skipping the exponentials of a
// wholly masked half was tried: the extra path in the loop cost 4-8 % and saved less.
template <int D>
struct Cfg {
    static constexpr int kColBlocks = D / 64;
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kKVBytes = 128 * D * 2;
    static constexpr int kStages = (D == 128) ? 5 : 8;
    static constexpr int kQOff = 0;
    static constexpr int kRingOff = 2 * kQBytes;
    static constexpr int kBarOff = kRingOff + kStages * kKVBytes;
    // full[S], empty[S], q_full[2], q_empty[2], s_full[3], p_full[2][3], pv_buf[3],
    // o_full, o_empty, drain[2], item_full[Q], item_empty[Q], v_tail[S], v_clean[S]
    static constexpr int kNumBars = 4 * kStages + 4 + kSBufs + 2 * kSBufs + kSBufs + 4 + 2 * kItemQ;
    static constexpr int kXchOff = kBarOff + kNumBars * 8;   // [2 halves][128 rows] fp32 exchange
    static constexpr int kMiscOff = kXchOff + 2 * 128 * 4;   // tmem base slot, abort flag
    static constexpr int kLostOff = kMiscOff + 16;           // kLostWords
    static constexpr int kQueueOff = kLostOff + 4 * packed::kLostWords;  // item queue
    static constexpr int kSmemBytes = kQueueOff + kItemQ * int(sizeof(QWork)) + 1024;
    static_assert(kQueueOff % 16 == 0, "queue entries are 16-byte aligned");
    __host__ __device__ static constexpr uint32_t col_s(int buf) { return uint32_t(buf) * 128u; }
    static constexpr uint32_t kColO = kSBufs * 128u;
    static_assert(kSBufs * 128 + D <= int(kTmemCols), "TMEM budget");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
packed_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const FwdParams p) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const uint32_t bar0 = base + C::kBarOff;
    constexpr int S = C::kStages;
    constexpr int NB = kSBufs;
    auto bar_full = [&](int r) { return bar0 + 8u * r; };
    auto bar_empty = [&](int r) { return bar0 + 8u * (S + r); };
    auto bar_q_full = [&](int b) { return bar0 + 8u * (2 * S + b); };
    auto bar_q_empty = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };
    auto bar_s_full = [&](int b) { return bar0 + 8u * (2 * S + 4 + b); };
    auto bar_p_full = [&](int h, int b) { return bar0 + 8u * (2 * S + 4 + NB + NB * h + b); };
    auto bar_pv_buf = [&](int b) { return bar0 + 8u * (2 * S + 4 + 3 * NB + b); };
    const uint32_t xb = bar0 + 8u * (2 * S + 4 + 4 * NB);
    const uint32_t bar_o_full = xb, bar_o_empty = xb + 8;
    auto bar_drain = [&](int h) { return xb + 16 + 8u * h; };
    auto bar_item_full = [&](int q) { return xb + 32 + 8u * q; };
    auto bar_item_empty = [&](int q) { return xb + 32 + 8u * (kItemQ + q); };
    // Hand-over of a V with rows to clear, one pair for each ring slot: the load thread arrives
    // on v_tail once it has issued the copy (so the slot's `full` is in that copy's phase and
    // the tail warp's wait means that copy), the tail warp on v_clean.  The slot is not filled
    // again before PV has waited for v_clean, so neither side can be a phase ahead.
    auto bar_v_tail = [&](int r) { return xb + 32 + 8u * (2 * kItemQ + r); };
    auto bar_v_clean = [&](int r) { return xb + 32 + 8u * (2 * kItemQ + S + r); };
    static_assert(4 * S + 4 + 4 * NB + 4 + 2 * kItemQ == C::kNumBars, "barrier count");
    float* xch = reinterpret_cast<float*>(smem + C::kXchOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    volatile uint32_t* lost = reinterpret_cast<volatile uint32_t*>(smem + C::kLostOff);
    QWork* item_q = reinterpret_cast<QWork*>(smem + C::kQueueOff);
    auto wait_bar = [&](uint32_t bar, uint32_t parity) {
        return wait_bar_limited(bar, parity, abort_flag, p.status, p.timeout_ns);
    };
    // The CTA's k-th item, copied out of the queue; its entry is then free for item k + kItemQ.
    auto take_item = [&](uint32_t k, QWork& w) -> bool {
        const int q = int(k % kItemQ);
        if (!wait_bar(bar_item_full(q), (k / kItemQ) & 1u)) return false;
        w = item_q[q];
        return true;
    };

    if (threadIdx.x == 0) {
        for (int r = 0; r < S; ++r) {
            ptx::mbar_init(bar_full(r), 1);
            ptx::mbar_init(bar_empty(r), 1);
            ptx::mbar_init(bar_v_tail(r), 1);
            ptx::mbar_init(bar_v_clean(r), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar_q_full(b), 1);
            ptx::mbar_init(bar_q_empty(b), 1);
            ptx::mbar_init(bar_drain(b), 1);
        }
        for (int b = 0; b < NB; ++b) {
            ptx::mbar_init(bar_s_full(b), 1);
            ptx::mbar_init(bar_p_full(0, b), 4);  // one arrival for each softmax warp of the half
            ptx::mbar_init(bar_p_full(1, b), 4);
            ptx::mbar_init(bar_pv_buf(b), 1);
        }
        ptx::mbar_init(bar_o_full, 1);
        ptx::mbar_init(bar_o_empty, 8);
        for (int q = 0; q < kItemQ; ++q) {
            ptx::mbar_init(bar_item_full(q), 1);
            ptx::mbar_init(bar_item_empty(q), kItemConsumers);
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
    }
    if (warp == kPvWarp) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
        ptx::tmem_relinquish();
    }
    ops::grid_wait();  // the lists
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int32_t K = p.kv_heads;
    // Ring entry of chunk c's K and V in a block of n chunks (the load order:
    // K(0), K(1), K(2), then V(i), K(i + 3) for i = 0, 1, ...).
    auto entry_k = [](uint32_t c) { return c < uint32_t(NB) ? c : 2u * c - uint32_t(NB - 1); };
    auto entry_v = [](uint32_t i, uint32_t n) { return i + uint32_t(NB) <= n ? uint32_t(NB) + 2u * i : n + i; };

    if (warp == kLoadWarp) {
        ptx::regs_dec<kRegsProducer>();
        if (p.self) self_items(p.prob, item_q, int32_t(blockIdx.x), int32_t(gridDim.x));
        if (lane == 0) {
            // ------------------------------------------------------------ load
            const int32_t n_items = p.self ? 0 : p.v.lists->w_q * K;
            uint32_t ring = 0;
            uint32_t q_loads[2] = {0u, 0u};
            bool ok = !p.prob.waits.inject || wait_bar(bar_drain(0), 0);  // (arrived at on the way out only)
            auto issue = [&](const CUtensorMap* m, int32_t head, int32_t row) -> bool {
                const int r = int(ring % S);
                if (ring >= uint32_t(S) && !wait_bar(bar_empty(r), ((ring / S) - 1) & 1u)) return false;
                ptx::mbar_arrive_expect_tx(bar_full(r), C::kKVBytes);
#pragma unroll
                for (int cb = 0; cb < C::kColBlocks; ++cb)
                    ops::tma_load_3d(base + C::kRingOff + r * C::kKVBytes + cb * kBoxBytes, m, bar_full(r), cb * 64, head,
                                     row);
                ++ring;
                return true;
            };
            // A CTA's first item is its own number; the others come from the counter.  Where items
            // are many (8 to a CTA: short ones), the counter's answer for item k + 2 and the walk of
            // item k + 1 are on their way while item k's copies are issued; where they are few, an
            // item is only taken when the one before is issued, so that longest-first levels the
            // CTAs.  (8192 causal tokens, 24 / 8 heads, d = 128, dK / dV: 730 us late, 905 early.)
            const bool early = !p.self && n_items >= 8 * int32_t(gridDim.x);
            auto next = [&] { return int32_t(gridDim.x) + atomicAdd(&p.v.lists->next_q, 1); };
            auto fetch = [&](int32_t u) {
                QWork w{};
                w.n = -1;
                if (u < n_items) {
                    w = p.v.qwalks[u / K];
                    w.hk = u % K;
                }
                return w;
            };
            int32_t u2 = early ? next() : 0;
            QWork w1 = p.self ? item_q[0] : fetch(int32_t(blockIdx.x));
            for (uint32_t k = 0; ok; ++k) {
                const int qe = int(k % kItemQ);
                if (k > 0 && p.self)
                    w1 = item_q[qe];  // (the last entry is an end)
                else if (k > 0 && !early)
                    w1 = fetch(next());
                const QWork q = w1;
                if (k >= uint32_t(kItemQ) && !wait_bar(bar_item_empty(qe), ((k / kItemQ) - 1) & 1u)) break;
                if (!p.self) item_q[qe] = q;
                ptx::mbar_arrive(bar_item_full(qe));
                if (q.n < 0) break;
                if (early) {
                    w1 = fetch(u2);
                    if (u2 < n_items) u2 = next();
                }
                const int32_t hk = q.hk, n = q.n, row0 = q.key0 + q.c0 * 128;
                const int qb = int(k & 1u);
                if (!wait_bar(bar_q_empty(qb), ((k >> 1) & 1u) ^ 1u)) break;
                ptx::mbar_arrive_expect_tx(bar_q_full(qb), C::kColBlocks * p.q_box_bytes);
#pragma unroll
                for (int cb = 0; cb < C::kColBlocks; ++cb)
                    ops::tma_load_3d(base + C::kQOff + qb * C::kQBytes + cb * kBoxBytes, &tm_q, bar_q_full(qb), cb * 64,
                                     hk * p.group, q.tok0);
                ++q_loads[qb];
                for (int32_t c = 0; ok && c < n && c < NB; ++c) ok = issue(&tm_k, hk, row0 + c * 128);
                for (int32_t i = 0; ok && i < n; ++i) {
                    ok = issue(&tm_v, hk, row0 + i * 128);
                    if (ok && i >= first_care(q)) ptx::mbar_arrive(bar_v_tail(int((ring - 1) % S)));
                    if (ok && i + NB < n) ok = issue(&tm_k, hk, row0 + (i + NB) * 128);
                }
            }
            // Drain the copies that may still be in flight (after an abort).
            const uint32_t first = ring > uint32_t(S) ? ring - S : 0u;
            for (uint32_t it = first; it < ring; ++it) drain_bar(bar_full(int(it % S)), (it / S) & 1u, p.timeout_ns);
            for (int b = 0; b < 2; ++b)
                if (q_loads[b] > 0) drain_bar(bar_q_full(b), (q_loads[b] - 1u) & 1u, p.timeout_ns);
        }
    } else if (warp == kTailWarp) {
        ptx::regs_dec<kRegsProducer>();
        if (p.self && p.prob.clear_tail) self_clear(p.prob, D, p.o, p.lse);
        // ------------------------------------------------------------ V tails
        uint32_t e0 = 0, tails = 0;  // tails, bit r: phase of slot r's v_tail
        for (uint32_t kq = 0;; ++kq) {
            QWork q;
            if (!__all_sync(~0u, take_item(kq, q))) break;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_item_empty(int(kq % kItemQ)));
            if (q.n < 0) break;
            const uint32_t n = uint32_t(q.n);
            bool ok = true;
            for (uint32_t i = uint32_t(first_care(q)); i < n; ++i) {
                const uint32_t e = e0 + entry_v(i, n);
                const int r = int(e % S);
                ok = __all_sync(~0u, wait_bar(bar_v_tail(r), (tails >> r) & 1u) && wait_bar(bar_full(r), (e / S) & 1u));
                if (!ok) break;
                tails ^= 1u << r;
                const int key = (q.c0 + int(i)) * 128, dead = dead_from(q, p.causal, key);
                uint8_t* v0 = smem + C::kRingOff + r * C::kKVBytes;
                for (int j = dead * 8 + lane; j < 128 * 8; j += 32)
#pragma unroll
                    for (int cb = 0; cb < C::kColBlocks; ++cb)
                        *reinterpret_cast<uint4*>(v0 + cb * kBoxBytes + j * 16) = make_uint4(0u, 0u, 0u, 0u);
                if (packed::scrub_rows<C::kColBlocks>(v0, kBoxBytes, hidden_from(q, key), dead, lane, 32))
                    lost[kq % packed::kLostWords] = kq + 1;
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_v_clean(r));
            }
            if (!ok) break;
            e0 += 2u * n;
        }
    } else if (warp == kPvWarp || warp == kSWarp) {
        ptx::regs_dec<kRegsProducer>();
        if (lane == 0) {
            // ------------------------------------------------------------- MMA
            const bool pv_role = warp == kPvWarp;
            constexpr uint32_t idesc_qk = ptx::idesc_bf16(128, 128, false);
            constexpr uint32_t idesc_pv = ptx::idesc_bf16(128, D, true);
            uint32_t e0 = 0, g = 0;
            uint32_t cleaned = 0;  // bit r: phase of slot r's v_clean
            bool ok = true;
            auto wait_entry = [&](uint32_t e, uint32_t& addr) -> bool {
                const int r = int(e % S);
                if (!wait_bar(bar_full(r), (e / S) & 1u)) return false;
                addr = base + C::kRingOff + r * C::kKVBytes;
                return true;
            };
            for (uint32_t kq = 0; ok; ++kq) {
                QWork q;
                if (!take_item(kq, q)) break;
                ptx::mbar_arrive(bar_item_empty(int(kq % kItemQ)));
                if (q.n < 0) break;
                const uint32_t n = uint32_t(q.n);
                const uint32_t g0 = g;
                if (pv_role) {
                    const uint32_t tO = tmem + C::kColO;
                    for (uint32_t i = 0; ok && i < n; ++i) {
                        const uint32_t gi = g0 + i, bb = gi % uint32_t(NB), e = e0 + entry_v(i, n);
                        uint32_t vaddr;
                        if (!wait_entry(e, vaddr)) { ok = false; break; }
                        if (i >= uint32_t(first_care(q))) {
                            const uint32_t r = e % S;
                            if (!wait_bar(bar_v_clean(int(r)), (cleaned >> r) & 1u)) { ok = false; break; }
                            cleaned ^= 1u << r;
                        }
                        if (i == 0 && !wait_bar(bar_o_empty, (kq & 1u) ^ 1u)) { ok = false; break; }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!wait_bar(bar_p_full(h, int(bb)), (gi / uint32_t(NB)) & 1u)) {
                                ok = false;
                                break;
                            }
                            ptx::tc_fence_after();
                            const uint32_t tP = tmem + C::col_s(int(bb)) + uint32_t(h) * 64u;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                ptx::mma_ts(tO, tP + kk * 8,
                                            ptx::desc_mn_sw128(vaddr + (h * 4 + kk) * 16 * 128, kBoxBytes), idesc_pv,
                                            (i > 0 || h > 0 || kk > 0) ? 1u : 0u);
                        }
                        if (!ok) break;
                        ptx::mma_commit(bar_pv_buf(int(bb)));
                        ptx::mma_commit(bar_empty(int(e % S)));
                    }
                    if (!ok) break;
                    ptx::mma_commit(bar_o_full);
                } else {
                    const int qb = int(kq & 1u);
                    const uint32_t qaddr = base + C::kQOff + qb * C::kQBytes;
                    if (!wait_bar(bar_q_full(qb), (kq >> 1) & 1u)) break;
                    for (uint32_t c = 0; ok && c < n; ++c) {
                        const uint32_t gc = g0 + c, bb = gc % uint32_t(NB), e = e0 + entry_k(c);
                        if (gc >= uint32_t(NB) && !wait_bar(bar_pv_buf(int(bb)), ((gc / uint32_t(NB)) - 1u) & 1u)) {
                            ok = false;
                            break;
                        }
                        uint32_t kaddr;
                        if (!wait_entry(e, kaddr)) { ok = false; break; }
                        ptx::tc_fence_after();
                        const uint32_t tS = tmem + C::col_s(int(bb));
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t coff = (kk >> 2) * kBoxBytes + (kk & 3) * 32;
                            ptx::mma_ss(tS, ptx::desc_k_sw128(qaddr + coff), ptx::desc_k_sw128(kaddr + coff), idesc_qk,
                                        kk > 0 ? 1u : 0u);
                        }
                        ptx::mma_commit(bar_s_full(int(bb)));
                        ptx::mma_commit(bar_empty(int(e % S)));
                    }
                    if (!ok) break;
                    ptx::mma_commit(bar_q_empty(qb));
                }
                g = g0 + n;
                e0 += 2u * n;
            }
            const int dr = pv_role ? 0 : 1;
            ptx::mma_commit(bar_drain(dr));
            drain_bar(bar_drain(dr), 0, p.timeout_ns);
        }
    } else {
        // ------------------------------------------------------------- softmax
        ptx::regs_inc<kRegsSoftmax>();
        const int half = warp >> 2;  // 0: keys 0-63 of every chunk, 1: keys 64-127
        const int row = threadIdx.x & 127;
        const uint32_t pair_bar = 1u + uint32_t(warp & 3);  // named barrier of warps w and w + 4
        const uint32_t lane_addr = uint32_t((warp & 3) * 32) << 16;
        const uint32_t tOh = tmem + lane_addr + C::kColO + uint32_t(half) * (D / 2);  // this half's O columns
        float* x_mine = xch + half * 128 + row;
        const float* x_other = xch + (1 - half) * 128 + row;
        const float c = p.scale_log2;
        const int r_tok = row / p.group, r_head = row - r_tok * p.group;
        uint32_t g = 0;
        bool ok = true;
        for (uint32_t kq = 0; ok; ++kq) {
            QWork q;
            q.n = -1;
            const bool took = __all_sync(~0u, take_item(kq, q));
            __syncwarp();
            if (took && lane == 0) ptx::mbar_arrive(bar_item_empty(int(kq % kItemQ)));
            if (ptx::bar_red_or(pair_bar, 64, !took)) {  // leave together
                ok = false;
                break;
            }
            if (q.n < 0) break;
            const uint32_t n = uint32_t(q.n);
            const bool real = r_tok < q.ntok;
            const int limit = real ? min(q.nkeys, q.limit0 + (p.causal ? r_tok : 0)) : INT32_MAX;
            const int warp_limit = __reduce_min_sync(~0u, limit);  // over the rows that are stored
            float m_used = 0.0f, l = 0.0f;
            uint32_t sr[64];
            bool pre = false;  // sr already holds S(g)
            for (uint32_t i = 0; i < n; ++i, ++g) {
                const uint32_t b = g % uint32_t(NB), b1 = (g + 1u) % uint32_t(NB);
                const uint32_t tS = tmem + lane_addr + C::col_s(int(b)) + uint32_t(half) * 64u;
                const uint32_t tS1 = tmem + lane_addr + C::col_s(int(b1)) + uint32_t(half) * 64u;
                bool wok = true;
                if (!pre) {
                    wok = __all_sync(~0u, wait_bar(bar_s_full(int(b)), (g / uint32_t(NB)) & 1u));
                    if (wok) {
                        ptx::tc_fence_after();
                        ptx::tmem_ld64(tS, sr);
                    }
                }
                pre = false;
                const int kbeg = (q.c0 + int(i)) * 128 + half * 64;
                const bool masked = kbeg + 64 > warp_limit;
                if (wok && masked) mask_from(sr, limit - kbeg);
                // Is S(g + 1) of this block complete?  If so, its load starts
                // right after the exponentials and overlaps the P hand-over.
                const bool can_pre = wok && i > 0 && i + 1 < n;
                const bool t_next =
                    can_pre && ptx::mbar_test_wait(bar_s_full(int(b1)), ((g + 1u) / uint32_t(NB)) & 1u);
                uint32_t pk[32];
                float rowsum = 0.0f;
                bool need = false;
                if (wok && i > 0) {
                    rowsum = softmax_exp64(sr, c, m_used, pk);  // against the running max (no max pass)
                    need = real && !(rowsum <= kRescaleRowSum);  // also catches inf
                }
                const bool nxt = can_pre && __all_sync(~0u, t_next);
                if (nxt) {
                    ptx::tc_fence_after();
                    ptx::tmem_ld64_start(tS1, sr);
                }
                if (ptx::bar_red_or(pair_bar, 64, !wok || need || i == 0)) {
                    // ---- slow path: the block's first chunk, a rescale, or an abort.
                    // Both warps of the pair take it, exchange this chunk's
                    // maxima of the rows that need it and agree on the new running max.
                    // (Of those alone: what a row comes to never depends on other rows.)
                    if (nxt) {
                        ptx::tmem_wait_ld(sr);
                        ptx::tmem_ld64(tS, sr);  // S(g) again: P(g) is not stored yet
                        if (masked) mask_from(sr, limit - kbeg);
                    }
                    *x_mine = wok && (need || i == 0) ? row_max64(sr) : -INFINITY;
                    if (ptx::bar_red_or(pair_bar, 64, !wok)) {
                        ok = false;
                        break;
                    }
                    const float mx = fmaxf(*x_mine, *x_other);
                    float alpha = 1.0f;
                    if (i == 0) {
                        m_used = mx == -INFINITY ? p.nothing_yet : mx;  // (no key, or scores of -inf alone)
                    } else if ((mx - m_used) * c > 0.0f) {
                        alpha = ptx::ex2((m_used - mx) * c);
                        m_used = mx;
                    }
                    rowsum = softmax_exp64(sr, c, m_used, pk);
                    ptx::tmem_st32(tS, pk);
                    l = l * alpha + rowsum;
                    bool pv_ok = true;
                    if (i > 0) {
                        // O holds P(.. g - 1) V: wait for PV(g - 1), the one that
                        // may still run, then rescale this half's columns of O.
                        const uint32_t gp = g - 1u;
                        pv_ok = __all_sync(~0u, wait_bar(bar_pv_buf(int(gp % uint32_t(NB))), (gp / uint32_t(NB)) & 1u));
                        if (pv_ok && __any_sync(~0u, alpha != 1.0f)) {
                            ptx::tc_fence_after();
                            const uint64_t alpha2 = ptx::f2(alpha, alpha);
#pragma unroll 1
                            for (int cb = 0; cb < D / 64; ++cb) {
                                uint32_t orr[32];
                                ptx::tmem_ld32(tOh + cb * 32, orr);
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    float o0, o1;
                                    ptx::f2_split(ptx::f2_mul(ptx::f2(__uint_as_float(orr[2 * j]),
                                                                      __uint_as_float(orr[2 * j + 1])), alpha2),
                                                  o0, o1);
                                    orr[2 * j] = __float_as_uint(o0);
                                    orr[2 * j + 1] = __float_as_uint(o1);
                                }
                                ptx::tmem_st32(tOh + cb * 32, orr);
                            }
                        }
                    }
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    // both halves' rescales of O are done before either half's P is signalled
                    if (ptx::bar_red_or(pair_bar, 64, !pv_ok)) {
                        ok = false;
                        break;
                    }
                    if (nxt) ptx::tmem_ld64(tS1, sr);  // S(g + 1) again
                } else {
                    ptx::tmem_st32(tS, pk);
                    l += rowsum;
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    if (nxt) ptx::tmem_wait_ld(sr);
                }
                pre = nxt;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_p_full(half, int(b)));
            }
            if (!ok) break;
            // ---- epilogue: O / (l_A + l_B) -> bf16, LSE; each half stores its columns.
            const bool ook = __all_sync(~0u, wait_bar(bar_o_full, kq & 1u));
            *x_mine = l;
            if (ptx::bar_red_or(pair_bar, 64, !ook)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const float l_sum = l + *x_other;
            const bool none = l_sum == 0.0f;  // no visible key: O = 0, whatever TMEM holds
            const float inv_l = 1.0f / l_sum;
            const uint64_t f2inv = ptx::f2(inv_l, inv_l);
            const int32_t head = q.hk * p.group + r_head;
            const int64_t tok = q.tok0 + r_tok;
            uint4* dst = reinterpret_cast<uint4*>(p.o.p + tok * p.o.ts + head * p.o.hs + half * (D / 2));
            // a part: O unnormalised in fp32, four columns of all rows after four columns (a warp's stores are
            // whole lines), and behind it of each row m (in units of log2) and l
            float* part = p.v.parts + (int64_t(q.slot) * K + q.hk) * (128 * (D + 2));
            const bool fix = real && lost[kq % packed::kLostWords] == kq + 1;
#pragma unroll 1
            for (int cb = 0; cb < D / 64; ++cb) {
                uint32_t orr[32];
                ptx::tmem_ld32(tOh + cb * 32, orr);  // every lane loads: the access is warp-wide
                if (fix) {
                    int lo;
                    const int seen = lost_seen(q, limit, lo);
                    packed::restore(orr, p.vals.p + (q.key0 + int64_t(lo)) * p.vals.ts + q.hk * p.vals.hs + half * (D / 2) + cb * 32,
                                    p.vals.ts, seen);
                }
                if (q.slot >= 0) {
                    float4* d4 = reinterpret_cast<float4*>(part) + (half * (D / 8) + cb * 8) * 128 + row;
                    if (real)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            d4[j * 128] = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                         : make_float4(__uint_as_float(orr[4 * j]), __uint_as_float(orr[4 * j + 1]),
                                                       __uint_as_float(orr[4 * j + 2]), __uint_as_float(orr[4 * j + 3]));
                    continue;
                }
                uint32_t pk[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float o0, o1;
                    ptx::f2_split(ptx::f2_mul(ptx::f2(__uint_as_float(orr[2 * j]), __uint_as_float(orr[2 * j + 1])),
                                              f2inv),
                                  o0, o1);
                    pk[j] = none ? 0u : ptx::pack_bf16x2(o0, o1);
                }
                if (real) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        dst[cb * 4 + j] = make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
                }
            }
            if (q.slot >= 0) {
                if (half == 0 && real)
                    *reinterpret_cast<float2*>(part + 128 * D + 2 * row) = make_float2(none ? -INFINITY : m_used * c, l_sum);
            } else if (half == 0 && real)
                p.lse[int64_t(head) * p.tokens_q + tok] = none ? -INFINITY : m_used * p.scale + logf(l_sum);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_o_empty);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kPvWarp) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

// No keys at all: every row of every sequence is empty.
__global__ void packed_no_keys_kernel(const PackedProblem p, const packed::View v, int head_dim, Rows o, float* lse) {
    ops::grid_wait();
    const int parts = head_dim / 8;
    for (int e = blockIdx.x; e < v.lists->n_q; e += gridDim.x) {
        const QBlock q = v.qblocks[e];
        for (int i = threadIdx.x; i < q.ntok * p.heads * parts; i += blockDim.x) {
            const int row = i / parts;
            const int64_t tok = q.tok0 + row / p.heads;
            const int h = row % p.heads;
            *reinterpret_cast<uint4*>(o.p + tok * o.ts + h * o.hs + (i % parts) * 8) = make_uint4(0u, 0u, 0u, 0u);
            if (lse != nullptr && i % parts == 0) lse[int64_t(h) * p.tokens_q + tok] = -INFINITY;
        }
    }
}

// Bound by latency (a few microseconds beside the launch); each part is read once.
// Joins the parts of split query blocks: O = sum 2^(m_i - m) O_i / l, in the order of the parts.
// Eight rows (of blockIdx.y) to a CTA, four columns of a row to a thread.
constexpr int kJoinRows = 8;
template <int D>
__global__ void __launch_bounds__(kJoinRows * D / 4) packed_join_kernel(const FwdParams p) {
    ops::grid_wait();
    const int K = p.kv_heads, row = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows, c4 = threadIdx.x / kJoinRows;
    const int64_t n = int64_t(p.v.lists->n_q) * K;
    for (int64_t w = blockIdx.x; w < n; w += gridDim.x) {
        const QBlock q = p.v.qblocks[w / K];
        const int hk = int(w % K);
        if (q.split < 2 || row >= q.ntok * p.group) continue;
        const float* part = p.v.parts + (int64_t(q.slot) * K + hk) * (128 * (D + 2));
        const int64_t step = int64_t(K) * (128 * (D + 2));
        float m = -INFINITY;
#pragma unroll 4
        for (int i = 0; i < q.split; ++i) m = fmaxf(m, part[i * step + 128 * D + 2 * row]);
        const float mu = m == -INFINITY ? 0.0f : m;
        float l = 0.0f, x[4] = {};
#pragma unroll 4
        for (int i = 0; i < q.split; ++i) {
            const float* src = part + i * step;
            const float2 st = *reinterpret_cast<const float2*>(src + 128 * D + 2 * row);
            const float4 o = reinterpret_cast<const float4*>(src)[c4 * 128 + row];
            const float f = ptx::ex2(st.x - mu);
            l += st.y * f;
            x[0] += o.x * f;
            x[1] += o.y * f;
            x[2] += o.z * f;
            x[3] += o.w * f;
        }
        const bool none = l == 0.0f;
        const float inv = none ? 0.0f : 1.0f / l;
        const int64_t tok = q.tok0 + row / p.group;
        const int head = hk * p.group + row % p.group;
        *reinterpret_cast<uint2*>(p.o.p + tok * p.o.ts + head * p.o.hs + c4 * 4) =
            none ? make_uint2(0u, 0u)
                 : make_uint2(ptx::pack_bf16x2(x[0] * inv, x[1] * inv), ptx::pack_bf16x2(x[2] * inv, x[3] * inv));
        if (c4 == 0) p.lse[int64_t(head) * p.tokens_q + tok] = none ? -INFINITY : (mu + log2f(l)) * 0.6931471805599453f;
    }
}

// Are the walks short enough for two items at a time (sta_packed_pair.cu)?  By the mean number of
// keys of a sequence; 16384 tokens, pair / one at a time, us: d = 128, 24 / 8 heads, causal, sequences
// of 256: 103 / 145, 512: 140 / 157, 768: 169 / 173, 1024: 203 / 195, 4096: 577 / 470; 24 / 24 heads, not causal,
// 512: 162 / 198, 1024: 294 / 297; d = 64, 16 / 2 heads, causal, 1024: 118 / 124, 2048: 193 / 180, 4096: 330 / 278.
bool short_walks(const PackedProblem& p, int head_dim) {
    return p.tokens_k <= int64_t(p.batch) * (head_dim == 128 ? 768 : 1500);
}

template <int D>
cudaError_t launch_fwd(const PackedProblem& p, const Rows& q, const Rows& k, const Rows& v, const Rows& o, float* lse,
                       const packed::Layout& w, const packed::View& view, bool self, cudaStream_t stream) {
    const int tpb = 128 / p.group;
    CUtensorMap mq, mk, mv;
    cudaError_t e = packed::rows_map(&mq, q, p.tokens_q, p.heads, D, p.group, tpb);
    if (e == cudaSuccess) e = packed::rows_map(&mk, k, p.tokens_k, p.kv_heads, D, 1, 128);
    if (e == cudaSuccess) e = packed::rows_map(&mv, v, p.tokens_k, p.kv_heads, D, 1, 128);
    if (e != cudaSuccess) return e;
    FwdParams fp{view, p, self ? 1 : 0, p.kv_heads, p.group, p.causal, p.tokens_q, o, v, lse, p.scale, p.scale * 1.4426950408889634f,
                 -3.0e38f / std::max(p.scale * 1.4426950408889634f, 1.0f),
                 uint32_t(p.group * tpb) * 128u, p.status, p.waits.timeout_ns};
    constexpr int kSmem = Cfg<D>::kSmemBytes;
    const int64_t items = w.max_wq * p.kv_heads;
    if (short_walks(p, D)) {
        e = packed_fwd::launch_forward_pair(D, mq, mk, mv, fp, items, w.sms, stream);
    } else {
        e = cudaFuncSetAttribute(packed_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess)
            e = packed::launch(packed_fwd_kernel<D>, dim3(unsigned(items < w.sms ? items : w.sms)), kThreads, kSmem, stream,
                               true, mq, mk, mv, fp);
    }
    if (e == cudaSuccess && !self && w.split_q) {
        const int64_t blocks = w.max_q * p.kv_heads;
        e = packed::launch(packed_join_kernel<D>, dim3(unsigned(blocks), 128 / kJoinRows), kJoinRows * D / 4, 0, stream, true, fp);  // (fewer than 2 SMs' worth)
    }
    return e;
}

// Takes one bit from the status word, the timeout's first: what other streams' kernels set meanwhile stays.
__global__ void take_status_kernel(uint32_t* word, uint32_t* taken) {
    const uint32_t now = atomicOr(word, 0u), bit = (now & kDevTimeout) != 0u ? uint32_t(kDevTimeout) : now & uint32_t(kDevBounds);
    atomicAnd(word, ~bit);
    *taken = bit;
}

// Does the forward plan this problem in the kernel?
bool self_planned(const PackedProblem& p, const packed::Layout& w) {
    return p.batch > 0 && p.batch <= kSelfBatch && p.tokens_k > 0 && !w.split_q &&
           w.max_q * p.kv_heads <= int64_t(kSelfItems) * w.sms;
}

}  // namespace

OpWaits op_waits() {
    const int32_t ms = g_op_inject_ms.load();  // 0: off
    return ms > 0 ? OpWaits{uint64_t(ms) * 1000000ull, 1} : OpWaits{kTimeoutNs, 0};
}

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
                         p->cu_q, p->cu_k, p->causal, p->clear_tail, p->softmax_scale, nullptr, op_waits()};
    return STA_OK;
}

cudaError_t launch_packed_forward(const PackedProblem& p, int head_dim, const Rows& q, const Rows& k, const Rows& v,
                                  const Rows& o, float* lse, void* workspace, cudaStream_t stream) {
    int sms = 0;
    if (cudaError_t e = packed::sm_count(&sms); e != cudaSuccess) return e;
    const packed::Layout w = packed::layout(p, false, head_dim, sms);
    const packed::View view = packed::view(w, workspace);
    if (self_planned(p, w)) {
        if (head_dim == 128) return launch_fwd<128>(p, q, k, v, o, lse, w, view, true, stream);
        return launch_fwd<64>(p, q, k, v, o, lse, w, view, true, stream);
    }
    packed::Tails tails{};
    tails.r[0] = o;
    tails.heads[0] = p.heads;
    tails.is_q[0] = 1;
    tails.n = 1;
    tails.lse = lse;
    const cudaError_t e = packed::launch_lists(p, view, false, head_dim, tails, stream);
    if (e != cudaSuccess || p.batch == 0) return e;
    if (p.tokens_k == 0)
        return packed::launch(packed_no_keys_kernel, dim3(unsigned(w.sms)), 256, 0, stream, true, p, view, head_dim, o, lse);
    if (head_dim == 128) return launch_fwd<128>(p, q, k, v, o, lse, w, view, false, stream);
    return launch_fwd<64>(p, q, k, v, o, lse, w, view, false, stream);
}

}  // namespace sta

using namespace sta;

extern "C" {

sta_status sta_packed_workspace(const sta_packed* p, int32_t backward, int64_t* bytes) {
    PackedProblem pp;
    if (bytes == nullptr || (backward != 0 && backward != 1)) return STA_ERR_INVALID_ARG;
    if (sta_status st = packed_problem(p, false, &pp); st != STA_OK) return st;
    const packed::Layout w = packed::layout(pp, backward != 0, p->head_dim, packed::sm_count_or_b200());
    *bytes = !backward && self_planned(pp, w) ? 0 : w.bytes;
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
    if (need > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || workspace_bytes < need))
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

sta_status sta_debug_inject_operator_timeout(int32_t mode, int32_t limit_ms) {
    if (mode < 0 || mode > 1 || limit_ms < 1 || limit_ms > 10000) return STA_ERR_INVALID_ARG;
    sta::g_op_inject_ms.store(mode == 1 ? limit_ms : 0);
    return STA_OK;
}

sta_status sta_operator_status(void* stream) {
    if (cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream)); e != cudaSuccess)
        return op_cuda_status(e);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return op_cuda_status(e);
    uint32_t* p = nullptr;
    if (cudaError_t e = op_status_word(&p); e != cudaSuccess) return op_cuda_status(e);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    void* taken = nullptr;
    uint32_t bit = 0;
    std::lock_guard<std::mutex> lock(g_taken_mutex);  // (one g_op_taken for each device)
    cudaError_t e = cudaGetSymbolAddress(&taken, g_op_taken);
    if (e == cudaSuccess) e = packed::launch(take_status_kernel, dim3(1), 1, 0, s, false, p, static_cast<uint32_t*>(taken));
    if (e == cudaSuccess) e = cudaMemcpyAsync(&bit, taken, sizeof bit, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return op_cuda_status(e);
    return bit == kDevTimeout ? STA_ERR_TIMEOUT : bit == kDevBounds ? STA_ERR_BOUNDS : STA_OK;
}

}  // extern "C"
