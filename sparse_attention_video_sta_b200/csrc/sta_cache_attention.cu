// sta_cache_attention.cu -- attention over the 8-bit paged cache.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "sta_ops.cuh"
#include "sta_ops.h"
#include "sta_packed.cuh"
#include "sta_ptx.cuh"
#include "sta_wait.cuh"

namespace sta {
namespace {

// Each warp streams tiles of 16 tokens through its own ring in shared memory and waits for
// another warp only at the end of its run.  A CTA has its SM alone (192 KB of rings: several
// times what 1 us of HBM latency needs).
constexpr int kTile = 16;      // tokens of a tile: in one block, whatever the block size
constexpr int kPlanWarps = 8;  // warps that sum the sequences
constexpr int kMostWarps = 12;
constexpr int kMinTiles = 4;   // a warp takes no fewer tiles, a CTA no fewer than two warps' worth
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -3.0e38f;  // running maximum of a row that has seen no key
constexpr float kRise = 8.0f;      // log2 by which a score may pass the running maximum before it is raised

// A unit, as its joins need it: its tiles, its first query token, the number of its rows, its
// first row of (token, head) and its first query head.  unit0 < 0: none.
struct Unit {
    int64_t unit0, unit1;
    int32_t q0, rows, row0, head;
};

struct CacheArgs {
    PackedProblem p;
    int32_t blocks, bt, bt_log2;
    int32_t row_tile;  // query rows of a unit
    const float* k_scales;
    const float* v_scales;
    const int32_t* lengths;
    const int32_t* tables;
    int32_t width;
    int64_t stride;
    Rows q, o;
    float* lse;
    float* warp_parts;  // [CTAs][warps][row_tile][D + 4]: O, m, l, mw
    float* cta_parts;   // [CTAs][2][row_tile][D + 4]
    Unit* begins;       // [CTAs]: the unit that a CTA's run begins inside of
    int64_t* head;      // tiles of all units, CTAs that take part
    uint64_t timeout_ns;
};

// The work: units of (sequence, `row_tile` query rows, key head), each of the sequence's tiles; all
// units' tiles in one row, cut into equal runs, one for each CTA, and those again, one for each
// warp.  A unit that lies in one warp's run is finished there; the parts of the others are
// joined by the CTA, and those of units that lie in several CTAs' runs by the second kernel,
// always in the order of the runs.
struct Sequence {
    int32_t q0, nq;      // its queries
    int32_t len, raw;    // tokens in the table; as given
    int32_t tiles;       // at least 1
    int32_t units;       // row tiles * key heads
};

// Bound i cut to the queries.
__device__ __forceinline__ int32_t bound(const CacheArgs& a, int i) { return max(0, min(a.p.cu_q[i], a.p.tokens_q)); }

// Sequence b; `top`: the largest bound before its own (0 will do where the bounds do not fall: they are
// made rising, as in the packed calls, so that no two sequences write the same rows).
__device__ __forceinline__ Sequence sequence(const CacheArgs& a, int b, int32_t top, bool* cut) {
    Sequence s;
    s.q0 = b;
    s.nq = 1;
    if (a.p.cu_q != nullptr) {
        const int32_t c0 = a.p.cu_q[b], c1 = a.p.cu_q[b + 1];
        s.q0 = max(top, min(c0, a.p.tokens_q));
        s.nq = max(s.q0, min(c1, a.p.tokens_q)) - s.q0;
        *cut |= c0 != s.q0 || c1 != s.q0 + s.nq;
    }
    s.raw = a.lengths[b];
    s.len = max(0, min(s.raw, a.width * a.bt));
    *cut |= s.raw != s.len;
    s.tiles = max(1, (s.len + kTile - 1) / kTile);
    s.units = (s.nq * a.p.group + a.row_tile - 1) / a.row_tile * a.p.kv_heads;
    return s;
}

struct PlanShared {
    int64_t scan[kPlanWarps];
    int64_t upto[kPlanWarps * 32];  // tiles of the sequences up to and with b (at most 256 sequences)
    int32_t first, last;  // the first sequence's first query, the end of the last one's queries
    int32_t tops[kPlanWarps];
    bool fall;        // a bound is below one before it
    int32_t top[kMostWarps];  // then each warp's, before its next sequence
};

// Inclusive maxima over a warp's lanes.
__device__ __forceinline__ int32_t warp_tops(int32_t v) {
    const int lane = threadIdx.x & 31;
    for (int i = 1; i < 32; i <<= 1) {
        const int32_t y = __shfl_up_sync(~0u, v, i);
        if (lane >= i) v = max(v, y);
    }
    return v;
}

// Bounds that fall (reported): this thread's tiles once more, the bounds made rising, 256 sequences at a time.
__device__ __forceinline__ int64_t plan_falling(const CacheArgs& a, PlanShared& sh) {
    const int warp = threadIdx.x / 32;
    int64_t n = 0;
    int32_t carry = 0;
    for (int b0 = 0; b0 < a.p.batch; b0 += kPlanWarps * 32) {
        const int b = b0 + int(threadIdx.x);
        const bool mine = warp < kPlanWarps && b < a.p.batch;
        int32_t top = warp_tops(mine ? bound(a, b) : 0);
        __syncthreads();
        if (warp < kPlanWarps && threadIdx.x % 32 == 31) sh.tops[warp] = top;
        __syncthreads();
        top = max(top, carry);
        for (int i = 0; i < kPlanWarps; ++i) {
            if (i < warp) top = max(top, sh.tops[i]);
            carry = max(carry, sh.tops[i]);
        }
        if (mine) {
            bool cut = false;
            const Sequence s = sequence(a, b, top, &cut);
            n += int64_t(s.tiles) * s.units;
        }
    }
    return n;
}

// The largest of the bounds before and of sequence b (one warp).
__device__ __forceinline__ int32_t top_upto(const CacheArgs& a, int b) {
    int32_t top = 0;
    for (int i = threadIdx.x & 31; i <= b; i += 32) top = max(top, bound(a, i));
    return __reduce_max_sync(~0u, top);
}

// Tiles of all units; the last query row.  (The first 8 warps sum; every thread calls.)
__device__ int64_t plan_total(const CacheArgs& a, PlanShared& sh, bool report) {
    int64_t n = 0;
    int32_t last = 0;
    bool cut = false;
    if (threadIdx.x == 0) {
        sh.first = sh.last = 0;
        sh.fall = false;
    }
    __syncthreads();
    if (threadIdx.x < kPlanWarps * 32)
        for (int b = threadIdx.x; b < a.p.batch; b += kPlanWarps * 32) {
            const Sequence s = sequence(a, b, 0, &cut);
            if (b == 0) {
                sh.first = s.q0;
                cut |= s.q0 != 0;
            }
            n += int64_t(s.tiles) * s.units;
            last = max(last, s.q0 + s.nq);
        }
    auto share = [&] {  // sums up to and with this thread in its warp; the warp's for the others
        const int lane = threadIdx.x & 31;
        for (int i = 1; i < 32; i <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, n, i);
            if (lane >= i) n += y;
        }
        if (lane == 31) sh.scan[threadIdx.x / 32] = n;
    };
    if (threadIdx.x < kPlanWarps * 32) {
        share();
        last = __reduce_max_sync(~0u, last);
        if (threadIdx.x % 32 == 0) atomicMax(&sh.last, last);
    }
    if (__syncthreads_or(cut)) {
        if (report && threadIdx.x == 0) atomicOr(a.p.status, kDevBounds);
        bool fall = false;
        if (a.p.cu_q != nullptr && threadIdx.x < kPlanWarps * 32)
            for (int b = threadIdx.x; b < a.p.batch; b += kPlanWarps * 32) fall |= bound(a, b + 1) < bound(a, b);
        if (__syncthreads_or(fall)) {
            if (threadIdx.x == 0) sh.fall = true;
            n = plan_falling(a, sh);
            if (threadIdx.x < kPlanWarps * 32) share();
            __syncthreads();
        }
    }
    int64_t total = 0;
    for (int i = 0; i < kPlanWarps; ++i) {
        if (i < int(threadIdx.x / 32)) n += sh.scan[i];
        total += sh.scan[i];
    }
    if (threadIdx.x < kPlanWarps * 32) sh.upto[threadIdx.x] = n;
    __syncthreads();
    return total;
}

// The sequence that holds tile `at`, and the tiles before it (one warp).
__device__ int32_t plan_locate(const CacheArgs& a, const PlanShared& sh, int64_t at, int64_t* before) {
    const int lane = threadIdx.x & 31;
    if (a.p.batch <= kPlanWarps * 32)
        for (int b0 = 0;; b0 += 32) {  // (upto does not fall, and its last is the total)
            const uint32_t past = __ballot_sync(~0u, sh.upto[b0 + lane] > at);
            if (past == 0u) continue;
            const int b = b0 + __ffs(past) - 1;
            *before = b == 0 ? 0 : sh.upto[b - 1];
            return b;
        }
    int64_t carry = 0;
    int32_t carry_top = 0;
    for (int b0 = 0;; b0 += 32) {
        bool cut = false;
        int64_t v = 0;
        int32_t top = 0;
        if (sh.fall) {
            top = max(carry_top, warp_tops(b0 + lane < a.p.batch ? bound(a, b0 + lane) : 0));
            carry_top = __shfl_sync(~0u, top, 31);
        }
        if (b0 + lane < a.p.batch) {
            const Sequence s = sequence(a, b0 + lane, top, &cut);
            v = int64_t(s.tiles) * s.units;
        }
        int64_t x = v;
        for (int i = 1; i < 32; i <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, x, i);
            if (lane >= i) x += y;
        }
        const uint32_t past = __ballot_sync(~0u, carry + x > at);
        if (past != 0u) {
            const int src = __ffs(past) - 1;
            *before = carry + __shfl_sync(~0u, x - v, src);
            return b0 + src;
        }
        carry += __shfl_sync(~0u, x, 31);
        if (b0 + 32 >= a.p.batch) return -1;  // (at is below the total: not reached)
    }
}

// One sequence alone: each of its units goes to a CTA where that leaves a warp at most so many tiles, and the
// second kernel has nothing to join (24 / 8 heads, d = 128, one query on 1000 tokens: 16.4 us joined, 14.1 so; on 1500:
// 17.1 / 16.2; with 12 on 2000: 17.0 / 18.7, on 2300: 15.3 / 19.9).
constexpr int kAlone = 8;
// CTAs that take part; the runs of the CTAs, or of a CTA's warps.
__device__ __forceinline__ int64_t plan_ctas(int64_t total, int64_t most) {
    const int64_t some = (total + 2 * kMinTiles - 1) / (2 * kMinTiles);
    return some < most ? some : most;
}
// n / d for n >= 0, d > 0: in 32 bits where they fit (a 64-bit division is some hundred instructions).
__device__ __forceinline__ int64_t divide(int64_t n, int32_t d) {
    return n <= int64_t(UINT32_MAX) ? int64_t(uint32_t(n) / uint32_t(d)) : n / d;
}
struct Runs {
    int64_t each, more;  // tiles of a run; the first `more` have one more
    __device__ Runs(int64_t total, int32_t parts) : each(divide(total, parts)), more(total - each * parts) {}
    __device__ int64_t first(int64_t i) const { return each * i + min(i, more); }
};

// D += A B, m16n8k16, fp16 operands, fp32 accumulators.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Bit 7 of each byte that is a NaN code of e4m3 (S.1111.111).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// 8 x 8 transpose of 16-bit values held two to a register across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Writes E of one row's outputs from `col` on, and its LSE.
template <int E>
__device__ __forceinline__ void store_row(const CacheArgs& a, int32_t tok, int32_t head, int col, const float* x, float m,
                                          float l, float mw) {
    const bool none = l == 0.0f;
    const float f = none ? 0.0f : ptx::ex2(mw - m) / l;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.o.p + int64_t(tok) * a.o.ts + head * a.o.hs + col);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) dst[i] = none ? 0u : ptx::pack_bf16x2(x[2 * i] * f, x[2 * i + 1] * f);
    if (col == 0) a.lse[int64_t(head) * a.p.tokens_q + tok] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Joins one row's n parts (part(c), c = 0 .. n - 1) in one warp: lane i returns columns
// i * D / 32 on of O in x, and m, l, mw.  Every share-th part from s on.
template <int D, class Part>
__device__ __forceinline__ void join_row(int64_t s, int64_t n, int share, const Part& part, float (&x)[D / 32], float& m,
                                         float& l, float& mw) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    m = mw = kNone;
    l = 0.0f;
    for (int64_t c = s + int64_t(lane) * share; c < n; c += 32 * share) {
        const float4 st = *reinterpret_cast<const float4*>(part(c) + D);
        m = fmaxf(m, st.x);
        mw = fmaxf(mw, st.z);
    }
    for (int k = 16; k > 0; k >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(~0u, m, k));
        mw = fmaxf(mw, __shfl_xor_sync(~0u, mw, k));
    }
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.0f;
#pragma unroll 8
    for (int64_t c = s; c < n; c += share) {
        const float* p = part(c);
        const float4 st = *reinterpret_cast<const float4*>(p + D);
        const float f = ptx::ex2(st.z - mw);
        l += st.y * ptx::ex2(st.x - m);
        if (E == 4) {
            const float4 y = *reinterpret_cast<const float4*>(p + lane * E);
            x[0] += y.x * f;
            x[1] += y.y * f;
            x[E - 2] += y.z * f;
            x[E - 1] += y.w * f;
        } else {
            const float2 y = *reinterpret_cast<const float2*>(p + lane * E);
            x[0] += y.x * f;
            x[1] += y.y * f;
        }
    }
}

// Attention over the cache, transposed: S^T = K Q^T and O^T += V^T W^T by mma.m16n8k16, tokens
// (then columns of V) as the 16 rows of an operand, 8 query rows as the columns.  A unit of 8
// rows (NT = 1: one token of up to 8 heads to a key head) then takes half the products and
// half the registers that rows-by-tokens would, and 16 rows (NT = 2) share one widening of the
// codes.  Operands are fp16 (the codes exactly, by cvt in registers: no widened copy
// anywhere), sums fp32.  Both products choose their summed index's order freely: K's 16 bytes
// of a thread are four k-steps, V's 16 bytes of two tokens are eight 2-row pieces of V^T after
// a byte interleave, and W^T is one movmatrix from S^T.
// A block's K scale multiplies the scores.  Its V scale 2^lv enters the exponent: W = 2^(S + lv - mw)
// with a running maximum mw of its own, so that W rounds to fp16 (2^-11 relative) relative to
// each row's largest contribution, however far the scales are apart; l sums the unscaled P
// = 2^(S - m) before any rounding.  Both maxima are raised only when a tile passes them by 2^8,
// which fp16 and fp32 bear and which makes rescaling O rare.  Q is scaled by a power of two
// for each row into fp16's range.
// HBM-bound: 2 D bytes for each token and key head.  64 requests of 500-8000 tokens, 24 / 8 heads, d = 128
// (313 MB): 72 us a call, 4.3 TB/s: the plan, the first copies' latency, the joins and 5.4 TB/s of
// 2 KB boxes between them (leaving the products out saved 7 of 77 us when it took that).
template <int D, int NT>
struct Cfg {
    static constexpr int kRows = 8 * NT;
    // O^T and Q^T take (D / 4 + D / 8) * NT registers: 12 warps of up to 168 where that is at most 48
    // (16 warps of 128 spill and take as long)
    static constexpr int kWarps = NT * D <= 128 ? 12 : 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kTileBytes = kTile * D;  // of K or V
    static constexpr int kStages = 192 * 1024 / (kWarps * 2 * kTileBytes) < 8 ? 192 * 1024 / (kWarps * 2 * kTileBytes) : 8;
    static constexpr int kRing = kWarps * kStages * 2 * kTileBytes;
    static constexpr int kBarOff = kRing;
    static constexpr int kSmem = kBarOff + kWarps * kStages * 8 + 1024;
    static_assert(kSmem <= 224 * 1024, "shared memory budget");
    static_assert(kWarps >= kPlanWarps && kWarps <= kMostWarps, "the plan's warps");
};

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1)
cache_attention_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const CacheArgs a) {
    using C = Cfg<D, NT>;
    constexpr int S = C::kStages, kWarps = C::kWarps, kThreads = C::kThreads, kRows = C::kRows;
    constexpr int kSteps = D / 16;    // k-steps of K Q^T, 16-row tiles of O^T
    extern __shared__ uint8_t smem_raw[];
    __shared__ PlanShared plan;
    __shared__ bool part0_kept[kWarps];  // in the ring
    __shared__ Unit ends[kWarps][2];  // each warp's parts: of the unit that it begins inside of, of its last
    const uint32_t raw_base = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int K = a.p.kv_heads, G = a.p.group;
    const uint32_t bar0 = base + C::kBarOff + warp * S * 8;
    uint8_t* ring = smem + warp * S * 2 * C::kTileBytes;
    if (lane == 0) {
        for (int i = 0; i < S; ++i) ptx::mbar_init(bar0 + 8u * i, 1);
        ptx::fence_barrier_init();
    }
    __syncwarp();
    ops::grid_launch_dependents();
    ops::grid_wait();

    const int64_t total = plan_total(a, plan, blockIdx.x == 0);
    if (a.p.clear_tail && plan.last - plan.first < a.p.tokens_q) {  // rows of no sequence
        const int32_t none = plan.first + a.p.tokens_q - plan.last, parts = D / 8;
        for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < int64_t(none) * a.p.heads * parts;
             i += int64_t(gridDim.x) * kThreads) {
            const int64_t row = i / parts;
            const int32_t nth = int32_t(row / a.p.heads), h = int32_t(row % a.p.heads);
            const int32_t tok = nth < plan.first ? nth : plan.last + nth - plan.first;
            *reinterpret_cast<uint4*>(a.o.p + tok * a.o.ts + h * a.o.hs + i % parts * 8) = make_uint4(0u, 0u, 0u, 0u);
            if (i % parts == 0) a.lse[int64_t(h) * a.p.tokens_q + tok] = -INFINITY;
        }
    }
    int64_t ctas = plan_ctas(total, gridDim.x);
    if (a.p.batch == 1) {  // a unit to a CTA, and nothing for the second kernel to join
        bool cut = false;
        const Sequence sq = sequence(a, 0, 0, &cut);
        if (sq.units > 0 && sq.units <= int64_t(gridDim.x) && sq.tiles <= kWarps * kAlone) ctas = sq.units;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.head[0] = total;
        a.head[1] = ctas;
    }
    if (blockIdx.x >= ctas) return;
    const Runs cta_runs(total, int32_t(ctas));
    const int64_t cta_begin = cta_runs.first(blockIdx.x), cta_end = cta_runs.first(blockIdx.x + 1);
    const int64_t n_tiles = cta_end - cta_begin, some = (n_tiles + kMinTiles - 1) / kMinTiles;
    const int warps = int(some < kWarps ? some : kWarps);  // that have a run
    const Runs runs(n_tiles, warps);
    const int64_t begin = cta_begin + (warp < warps ? runs.first(warp) : n_tiles);
    const int64_t end = cta_begin + (warp < warps ? runs.first(warp + 1) : n_tiles);
    if (lane < 2) ends[warp][lane].unit0 = -1;
    __syncwarp();
    // A part of what a run ends with stays in the warp's ring, which no copy fills any more; one of a unit
    // that ends inside of the run goes to the workspace.
    static_assert(S * 2 * C::kTileBytes >= kRows * (D + 4) * 4, "a part fits into a ring");
    float* my_part0 = a.warp_parts + (int64_t(blockIdx.x) * kWarps + warp) * kRows * (D + 4);
    int64_t at = begin, before = 0;
    int32_t b = at < end ? plan_locate(a, plan, at, &before) : 0;
    if (plan.fall && at < end) {
        const int32_t top = top_upto(a, b);
        if (lane == 0) plan.top[warp] = top;
        __syncwarp();
    }
    uint32_t slot_in = 0, slot_out = 0, phase = 0;  // this warp's ring: next slot to fill, to read, its phase
    uint32_t in_flight = 0;
    bool dead = false;

    while (at < end) {
        bool cut = false;
        const Sequence sq = sequence(a, b, plan.fall ? plan.top[warp] : 0, &cut);
        const int64_t in_seq = at - before;
        if (in_seq >= int64_t(sq.tiles) * sq.units) {
            before += int64_t(sq.tiles) * sq.units;
            ++b;
            if (plan.fall) {
                __syncwarp();
                if (lane == 0) plan.top[warp] = sq.q0 + sq.nq;
                __syncwarp();
            }
            continue;
        }
        const int unit = int(divide(in_seq, sq.tiles)), first = int(in_seq - int64_t(unit) * sq.tiles);
        const int rt = unit / K, hk = unit % K;
        const int last = int(min(int64_t(sq.tiles), first + (end - at)));
        at += last - first;
        const int t0 = first, t1 = last;
        const int rows = min(kRows, sq.nq * G - rt * kRows);
        // keys that row r sees: the first raw - nq + token + 1; never more than the table holds
        const uint32_t uG = uint32_t(G);  // (an unsigned division is half a signed one's instructions)
        auto limit_of = [&](int r) { return min(sq.len, sq.raw - sq.nq + int(uint32_t(rt * kRows + r) / uG) + 1); };
        const int least = limit_of(0);  // the smallest limit of the rows

        // ---- pages: lane i holds page `p0 + i` of the warp's run; the copies run ahead of the tiles, so the
        // tiles' scales have a window of their own (and the copies do not wait for them)
        const int pages = (min(sq.len, t1 * kTile) + a.bt - 1) >> a.bt_log2;
        const int32_t* table = a.tables + int64_t(b) * a.stride;
        auto page = [&](int from, bool report) {  // block of page from + lane; -1: none, or not in the pool
            const int j = from + lane;
            int id = j < pages ? table[j] : -1;
            if (j < pages && (id < 0 || id >= a.blocks)) {
                if (report) atomicOr(a.p.status, kDevBounds);
                id = -1;
            }
            return id;
        };
        int p0 = t0 * kTile >> a.bt_log2, s0 = p0;
        const int id0 = page(p0, true);
        int page_row = (max(id0, 0) * K + hk) << a.bt_log2;  // of the tensor maps; nothing is seen of a page that is not
        auto issue = [&](int tile) {
            const int tok = tile * kTile, pg = tok >> a.bt_log2;
            if (pg >= p0 + 32) {
                p0 = pg;
                page_row = (max(page(pg, true), 0) * K + hk) << a.bt_log2;
            }
            const int row = __shfl_sync(~0u, page_row, pg - p0) + (tok & (a.bt - 1));
            if (lane == 0) {
                const uint32_t bar = bar0 + 8u * slot_in, dst = ptx::smem_u32(ring + slot_in * 2 * C::kTileBytes);
                ptx::mbar_arrive_expect_tx(bar, 2 * C::kTileBytes);
                ptx::tma_load_2d(dst, &tm_k, bar, 0, row);
                if (!a.p.waits.inject)  // (debug: the tile never comes)
                    ptx::tma_load_2d(dst + C::kTileBytes, &tm_v, bar, 0, row);
            }
            slot_in = slot_in + 1 == S ? 0 : slot_in + 1;
            ++in_flight;
        };
        float page_ks, page_lv;  // ks < 0: not to be seen
        auto load_scales = [&](int id) {
            page_ks = id >= 0 ? a.k_scales[int64_t(id) * K + hk] : -1.0f;
            page_lv = id >= 0 ? a.v_scales[int64_t(id) * K + hk] : 1.0f;  // (its logarithm is taken when it is here)
        };
        // the queries' loads go out first, the first copies while they are on their way
        uint4 q_raw[NT][D / 32];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + g, row = rt * kRows + r;
            const bool have = r < rows;
            const uint32_t tok = have ? uint32_t(row) / uG : 0u, head = have ? uint32_t(row) - tok * uG : 0u;
            const __nv_bfloat16* src = a.q.p + int64_t(sq.q0 + int(tok)) * a.q.ts + (hk * G + int(head)) * a.q.hs;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                q_raw[nt][i] = make_uint4(0u, 0u, 0u, 0u);
                if (have) q_raw[nt][i] = __ldg(reinterpret_cast<const uint4*>(src + (t + 4 * (i >> 1)) * 16 + (i & 1) * 8));
            }
        }
        load_scales(id0);
        int next = t0;
        for (; next < t1 && next < t0 + S; ++next) issue(next);

        // ---- Q^T as the B operand of every k-step: thread (g, t) holds the 16-element pieces t, t + 4 of row g
        uint32_t qb[NT][kSteps][2];
        float rf[NT][2];    // factor of the products of rows 2t, 2t + 1
        int limit[NT][2];   // keys that they see
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t raw[D / 8];
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                raw[4 * i + 0] = q_raw[nt][i].x;
                raw[4 * i + 1] = q_raw[nt][i].y;
                raw[4 * i + 2] = q_raw[nt][i].z;
                raw[4 * i + 3] = q_raw[nt][i].w;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i) top = fmaxf(top, fmaxf(fabsf(bf_lo(raw[i])), fabsf(bf_hi(raw[i]))));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            // 2^e with |q| 2^e < 512: fp16 keeps elements down to 2^-33 of the largest
            const int e = min(max(8 - (int(__float_as_uint(top) >> 23) - 126), -119), 126);
            const float sc = __uint_as_float(uint32_t(e + 127) << 23);
            const float f = a.p.scale * kLog2e * __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                qb[nt][i][0] = half2_of(bf_lo(raw[2 * i]) * sc, bf_hi(raw[2 * i]) * sc);
                qb[nt][i][1] = half2_of(bf_lo(raw[2 * i + 1]) * sc, bf_hi(raw[2 * i + 1]) * sc);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                rf[nt][i] = __shfl_sync(~0u, f, (2 * t + i) * 4);
                limit[nt][i] = nt * 8 + 2 * t + i < rows ? limit_of(nt * 8 + 2 * t + i) : INT32_MAX;
            }
        }

        page_lv = log2f(page_lv);
        float o[NT][kSteps][4];
        float m[NT][2], mw[NT][2], l[NT][2], f[NT][2];  // of rows 2t, 2t + 1; f = 2^(m + lv - mw)
        float lv_now = 0.0f;                            // the lv that f holds for
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[nt][i] = mw[nt][i] = kNone;
                l[nt][i] = 0.0f;
                f[nt][i] = 1.0f;
            }
        }

        for (int tile = t0; tile < t1; ++tile) {
            const uint32_t bar = bar0 + 8u * slot_out;
            if (!__all_sync(~0u, ptx::mbar_try_wait(bar, phase))) {
                const uint64_t from = ptx::globaltimer_ns();
                for (int tries = 0; !ptx::mbar_try_wait(bar, phase); ++tries)
                    if (tries % 64 == 63 && ptx::globaltimer_ns() - from > a.timeout_ns) {
                        dead = true;  // give up waiting; the results are lost and reported
                        if (lane == 0) atomicOr(a.p.status, kDevTimeout);
                        break;
                    }
                if (__any_sync(~0u, dead)) {  // the warp stops together, and issues no more
                    dead = true;
                    break;
                }
            }
            const uint8_t* kt = ring + slot_out * 2 * C::kTileBytes;
            const uint8_t* vt = kt + C::kTileBytes;
            // ---- S^T = K Q^T (two sums over the k-steps, for a shorter chain)
            float s[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) s[nt][i][0] = s[nt][i][1] = s[nt][i][2] = s[nt][i][3] = 0.0f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint4 u[2];  // tokens g, g + 8 (rows of the swizzle differ by 8: the same chunk)
                const int chunk = t + 4 * c;
                const int off = D == 128 ? g * 128 + ((chunk ^ g) << 4) : g * 64 + ((chunk ^ ((g >> 1) & 3)) << 4);
                u[0] = *reinterpret_cast<const uint4*>(kt + off);
                u[1] = *reinterpret_cast<const uint4*>(kt + off + 8 * D);
                const uint32_t w0[4] = {u[0].x, u[0].y, u[0].z, u[0].w}, w1[4] = {u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t ka[4] = {ops::e4m3_half2(uint16_t(w0[q])), ops::e4m3_half2(uint16_t(w1[q])),
                                            ops::e4m3_half2(uint16_t(w0[q] >> 16)), ops::e4m3_half2(uint16_t(w1[q] >> 16))};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(s[nt][q & 1], ka, qb[nt][c * 4 + q][0], qb[nt][c * 4 + q][1]);
                }
            }
            // ---- scores in units of log2 (tokens g, g + 8; rows 2t, 2t + 1); masks
            const int tok = tile * kTile, pg = tok >> a.bt_log2;
            if (pg >= s0 + 32) {
                s0 = pg;
                load_scales(page(pg, false));
                page_lv = log2f(page_lv);
            }
            float2 mt;
            mt.x = __shfl_sync(~0u, page_ks, pg - s0);
            mt.y = __shfl_sync(~0u, page_lv, pg - s0);
            const bool masked = tok + kTile > least || mt.x < 0.0f;
            bool rise = false;
            float x[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nt][0][i] = (s[nt][0][i] + s[nt][1][i]) * (rf[nt][i & 1] * mt.x);
                if (masked)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (mt.x < 0.0f || tok + g + (i >> 1) * 8 >= limit[nt][i & 1]) s[nt][0][i] = -INFINITY;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    x[nt][i] = fmaxf(s[nt][0][i], s[nt][0][i + 2]);
                    rise |= x[nt][i] > m[nt][i] + kRise || x[nt][i] + mt.y > mw[nt][i] + kRise;
                }
            }
            if (__any_sync(~0u, rise)) {
                // raise the maxima of the rows that need it to this tile's, and rescale (of those alone: what a row
                // comes to does not depend on other rows)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int k = 4; k <= 16; k <<= 1) x[nt][i] = fmaxf(x[nt][i], __shfl_xor_sync(~0u, x[nt][i], k));
                        const bool up = x[nt][i] > m[nt][i] + kRise || x[nt][i] + mt.y > mw[nt][i] + kRise;
                        const float mn = up ? fmaxf(m[nt][i], x[nt][i]) : m[nt][i];
                        const float wn = up ? fmaxf(mw[nt][i], x[nt][i] + mt.y) : mw[nt][i];
                        const float cf = ptx::ex2(mw[nt][i] - wn);
                        l[nt][i] *= ptx::ex2(m[nt][i] - mn);
                        m[nt][i] = mn;
                        mw[nt][i] = wn;
#pragma unroll
                        for (int j = 0; j < kSteps; ++j) {
                            o[nt][j][i] *= cf;
                            o[nt][j][i + 2] *= cf;
                        }
                    }
                lv_now = INFINITY;  // f is stale
            }
            if (mt.y != lv_now) {
                lv_now = mt.y;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)  // where the factor is past fp32, P is 0
#pragma unroll
                    for (int i = 0; i < 2; ++i) f[nt][i] = ptx::ex2(fminf(m[nt][i] + mt.y - mw[nt][i], 126.0f));
            }
            uint32_t wb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = ptx::ex2(s[nt][0][i] - m[nt][i & 1]);
                l[nt][0] += p[0] + p[2];
                l[nt][1] += p[1] + p[3];
                wb[nt][0] = transpose8x8(half2_of(p[0] * f[nt][0], p[1] * f[nt][1]));
                wb[nt][1] = transpose8x8(half2_of(p[2] * f[nt][0], p[3] * f[nt][1]));
            }
            // ---- O^T += V^T W^T; thread (g, t) takes tokens 2t, 2t + 1, 2t + 8, 2t + 9 and the D / 8 columns
            // from g * D / 8 on
            uint32_t v[4][D / 32];  // [token][words]
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 2 * t + (i & 1) + (i >> 1) * 8;
                if (D == 128) {
                    const uint4 u = *reinterpret_cast<const uint4*>(vt + row * 128 + ((g ^ (row & 7)) << 4));
                    v[i][0] = u.x;
                    v[i][1] = u.y;
                    v[i][D / 32 - 2] = u.z;
                    v[i][D / 32 - 1] = u.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(vt + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) +
                                                                    (g & 1) * 8);
                    v[i][0] = u.x;
                    v[i][1] = u.y;
                }
                // what lies behind the last token (or in a block not to be seen) may be anything: 0 x NaN
                if (masked && (tok + row >= sq.len || mt.x < 0.0f))
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) v[i][j] = 0u;
            }
            __syncwarp();  // every lane has read the slot
            slot_out = slot_out + 1 == S ? 0 : slot_out + 1;
            phase ^= slot_out == 0 ? 1u : 0u;
            --in_flight;
            if (next < t1) issue(next++);
            if (masked) {
                // NaN codes in a tile that not every row sees whole: out of the products; another product counts for
                // each sum those that its row does see
                uint32_t bad[4][D / 32], any = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) any |= bad[i][j] = nan_codes(v[i][j]) >> 7;  // 1 in their bytes
                if (__any_sync(~0u, any != 0u)) {
#pragma unroll
                    for (int j = 0; j < D / 32; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            constexpr uint32_t kOne = 0x38;  // 1.0 in e4m3
                            const uint32_t sel = h == 0 ? 0x5140u : 0x7362u;
                            const uint32_t lo = __byte_perm(bad[0][j], bad[1][j], sel) * kOne,
                                           hi = __byte_perm(bad[2][j], bad[3][j], sel) * kOne;
                            const uint32_t is_nan[4] = {ops::e4m3_half2(uint16_t(lo)), ops::e4m3_half2(uint16_t(lo >> 16)),
                                                        ops::e4m3_half2(uint16_t(hi)), ops::e4m3_half2(uint16_t(hi >> 16))};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                auto sees = [&](int i) { return tok + g + (i >> 1) * 8 < limit[nt][i & 1] ? 1.0f : 0.0f; };
                                float count[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                mma16816(count, is_nan, transpose8x8(half2_of(sees(0), sees(1))),
                                         transpose8x8(half2_of(sees(2), sees(3))));
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (count[i] > 0.0f) o[nt][2 * j + h][i] = __uint_as_float(0x7fc00000u);
                            }
                        }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) v[i][j] &= ~(bad[i][j] * 0xffu);
                }
            }
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sel = h == 0 ? 0x5140u : 0x7362u;
                    const uint32_t lo = __byte_perm(v[0][j], v[1][j], sel), hi = __byte_perm(v[2][j], v[3][j], sel);
                    const uint32_t va[4] = {ops::e4m3_half2(uint16_t(lo)), ops::e4m3_half2(uint16_t(lo >> 16)),
                                            ops::e4m3_half2(uint16_t(hi)), ops::e4m3_half2(uint16_t(hi >> 16))};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][2 * j + h], va, wb[nt][0], wb[nt][1]);
                }
        }

        if (dead) break;
        // ---- the unit's rows (thread (g, t): D / 8 columns from g * D / 8 on, of rows 2t, 2t + 1)
        const bool whole = first == 0 && last == sq.tiles;
        const int64_t unit0 = at - last;  // the unit's first tile
        const int which = first > 0 ? 0 : 1;  // began in an earlier run (then this is the run's first), or here
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int k = 4; k <= 16; k <<= 1) l[nt][i] += __shfl_xor_sync(~0u, l[nt][i], k);
                const int r = nt * 8 + 2 * t + i;
                if (r >= rows) continue;
                float y[D / 8];
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
                    y[2 * j] = o[nt][j][i];
                    y[2 * j + 1] = o[nt][j][i + 2];
                }
                if (whole) {
                    const int row = rt * kRows + r;
                    store_row<D / 8>(a, sq.q0 + row / G, hk * G + row % G, g * (D / 8), y, m[nt][i], l[nt][i], mw[nt][i]);
                } else {
                    float* dst = (at == end ? reinterpret_cast<float*>(ring) : my_part0) + r * (D + 4);
#pragma unroll
                    for (int j = 0; j < D / 32; ++j)
                        *reinterpret_cast<float4*>(dst + g * (D / 8) + 4 * j) =
                            make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
                    if (g == 0) *reinterpret_cast<float4*>(dst + D) = make_float4(m[nt][i], l[nt][i], mw[nt][i], 0.0f);
                }
            }
        if (lane == 0 && !whole) ends[warp][which] = Unit{unit0, unit0 + sq.tiles, sq.q0, rows, rt * kRows, hk * G};
        if (lane == 0 && which == 0) part0_kept[warp] = at == end;
    }
    // After a wait that ran out: the copies still in flight land before the CTA leaves (bounded).
    if (dead)
        for (; in_flight > 0; --in_flight) {
            drain_bar(bar0 + 8u * slot_out, phase, a.timeout_ns);
            slot_out = slot_out + 1 == S ? 0 : slot_out + 1;
            phase ^= slot_out == 0 ? 1u : 0u;
        }
    // ---- the CTA's joins: of the unit that its run begins inside of, then of each unit that
    // begins inside of a warp's run and does not end there
    if (__syncthreads_or(dead)) {
        if (threadIdx.x == 0) a.begins[blockIdx.x].unit0 = -1;  // nothing for the second kernel to join from here
        return;
    }
    // (one warp for each row of each such unit)
    const float* parts0 = a.warp_parts + int64_t(blockIdx.x) * kWarps * kRows * (D + 4);
    // lane i < warps: does warp i's run begin inside of a unit, does it leave one unfinished
    const int64_t began = lane < warps ? ends[lane][0].unit0 : -1, left = lane < warps ? ends[lane][1].unit0 : -1;
    const uint32_t starts = __ballot_sync(~0u, left >= 0) << 1 | (__shfl_sync(~0u, began, 0) >= 0 ? 1u : 0u);
    int turn = 0;
    for (uint32_t todo = starts; todo != 0u; todo &= todo - 1) {
        const int w = __ffs(todo) - 2;  // -1: the unit that the CTA's run begins inside of
        const bool early = w < 0;
        const Unit u = early ? ends[0][0] : ends[w][1];
        const int w0 = early ? 0 : w;
        // the following runs that begin inside of the same unit
        const uint32_t same = __ballot_sync(~0u, began == u.unit0) >> (w0 + 1);
        const int w1 = w0 + __ffs(~same);
        const bool done = !early && u.unit1 <= cta_end;
        for (int r = 0; r < u.rows; ++r, ++turn) {
            if (turn % kWarps != warp) continue;
            float x[D / 32], jm, jl, jw;
            join_row<D>(0, w1 - w0, 1, [&](int64_t c) {
                const int v = w0 + int(c);
                const float* from = (c == 0 && !early) || part0_kept[v]
                                        ? reinterpret_cast<const float*>(smem + v * S * 2 * C::kTileBytes)
                                        : parts0 + int64_t(v) * kRows * (D + 4);
                return from + r * (D + 4);
            }, x, jm, jl, jw);
            if (done) {
                const int row = u.row0 + r;
                store_row<D / 32>(a, u.q0 + row / G, u.head + row % G, lane * (D / 32), x, jm, jl, jw);
            } else {
                float* dst = a.cta_parts + ((int64_t(blockIdx.x) * 2 + (early ? 0 : 1)) * kRows + r) * (D + 4);
#pragma unroll
                for (int e = 0; e < D / 32; ++e) dst[lane * (D / 32) + e] = x[e];
                if (lane == 0) *reinterpret_cast<float4*>(dst + D) = make_float4(jm, jl, jw, 0.0f);
            }
        }
    }
    if (threadIdx.x == 0) a.begins[blockIdx.x] = ends[0][0];
}

// Joins the parts of the units that lie in several CTAs' runs: one CTA here for each run that
// begins inside of a unit, if it is the first such run of its unit.  The parts: what the run
// before has of its last unit, then what this and the following runs have of their first.
constexpr int kJoinWarps = 32;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) cache_join_kernel(const CacheArgs a) {
    constexpr int E = D / 32;
    __shared__ alignas(16) float sh[kJoinWarps * (D + 4)];
    ops::grid_wait();
    const int64_t i = int64_t(blockIdx.x) + 1;
    const int64_t total = a.head[0], ctas = a.head[1];
    const Unit u = a.begins[i];  // (on its way with the others)
    if (i >= ctas) return;
    const Runs runs(total, int32_t(ctas));
    if (u.unit0 < 0 || runs.first(i - 1) > u.unit0) return;
    int64_t lo = i + 1, hi = ctas;  // the first CTA from i + 1 on whose run begins behind the unit
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (runs.first(mid) < u.unit1)
            lo = mid + 1;
        else
            hi = mid;
    }
    // a row for each warp, or (few rows) for each `share` warps, every one a share of the parts
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n = lo - i + 1;
    int share = 1;
    while (2 * share * u.rows <= kJoinWarps && 4 * share <= n) share *= 2;
    const int r = warp / share, s = warp % share;  // (units have at most 16 rows)
    float x[E], m, l, mw;
    if (r < u.rows) {
        join_row<D>(s, n, share, [&](int64_t c) {
            return a.cta_parts + ((c == 0 ? 2 * (i - 1) + 1 : 2 * (i + c - 1)) * a.row_tile + r) * (D + 4);
        }, x, m, l, mw);
        if (share > 1) {
            float* mine = sh + warp * (D + 4);
#pragma unroll
            for (int e = 0; e < E; ++e) mine[lane * E + e] = x[e];
            if (lane == 0) *reinterpret_cast<float4*>(mine + D) = make_float4(m, l, mw, 0.0f);
        }
    }
    __syncthreads();
    if (r >= u.rows || s > 0) return;
    if (share > 1) join_row<D>(0, share, 1, [&](int64_t c) { return sh + (warp + c) * (D + 4); }, x, m, l, mw);
    const int row = u.row0 + r;
    store_row<E>(a, u.q0 + row / a.p.group, u.head + row % a.p.group, lane * E, x, m, l, mw);
}

// Map over the codes as rows of D bytes; a box is `rows` of them, 128- or 64-byte swizzle.
cudaError_t codes_map(CUtensorMap* m, const void* codes, int64_t n_rows, int d, int rows) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static cudaError_t err = cudaSuccess;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        err = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q);
        if (err == cudaSuccess && q != cudaDriverEntryPointSuccess) err = cudaErrorNotSupported;
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    if (err != cudaSuccess) return err;
    cuuint64_t dims[2] = {cuuint64_t(d), cuuint64_t(n_rows)};
    cuuint64_t strides[1] = {cuuint64_t(d)};
    cuuint32_t box[2] = {cuuint32_t(d), cuuint32_t(rows)};
    cuuint32_t estr[2] = {1, 1};
    const CUresult c = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return c == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int NT>
cudaError_t launch_attention(const sta_cache& c, CacheArgs a, int sms, cudaStream_t stream) {
    using C = Cfg<D, NT>;
    const int64_t n_rows = int64_t(c.blocks) * c.kv_heads * c.block_tokens;
    CUtensorMap mk, mv;
    a.row_tile = C::kRows;
    a.cta_parts = a.warp_parts + int64_t(sms) * C::kWarps * C::kRows * (D + 4);
    a.begins = reinterpret_cast<Unit*>(a.cta_parts + int64_t(sms) * 2 * C::kRows * (D + 4));
    a.head = reinterpret_cast<int64_t*>(a.begins + sms);
    cudaError_t e = codes_map(&mk, c.k_codes, n_rows, D, kTile);
    if (e == cudaSuccess) e = codes_map(&mv, c.v_codes, n_rows, D, kTile);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(cache_attention_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e == cudaSuccess)
        e = packed::launch(cache_attention_kernel<D, NT>, dim3(unsigned(sms)), C::kThreads, C::kSmem, stream, true, mk, mv, a);
    if (e == cudaSuccess && sms > 1)
        e = packed::launch(cache_join_kernel<D>, dim3(unsigned(sms - 1)), kJoinWarps * 32, 0, stream, true, a);
    return e;
}

// Query rows of a unit, from the mean number of rows that a sequence has (its own are known
// on the device only): units of 16 rows widen the codes once for both halves.  (Units of 32
// leave 8 warps of 250 registers: 7 requests of 3000-30000 tokens with 1-6 drafted ones,
// 16 / 2 heads, d = 64, took 54 us, units of 16 took 41 then and take 36 now.)
template <int D>
cudaError_t launch_attention(const sta_cache& c, const CacheArgs& a, int sms, cudaStream_t stream) {
    const int64_t rows = a.p.batch > 0 ? int64_t(a.p.tokens_q) * a.p.group / a.p.batch : 0;
    return rows <= 8 ? launch_attention<D, 1>(c, a, sms, stream) : launch_attention<D, 2>(c, a, sms, stream);
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
    // tokens of the pool are int32 rows of the tensor maps
    if (int64_t(c->blocks) * c->kv_heads > INT32_MAX / c->block_tokens) return STA_ERR_UNSUPPORTED;
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
    const int sms = packed::sm_count_or_b200();
    // parts of an SM: its warps' (12 of 8 rows, 8 of 16; d = 64: 12 of 16) and its own two
    const int64_t rows = (c->head_dim == 128 ? 128 : 192) + 2 * 16;
    *bytes = sms * (rows * (c->head_dim + 4) * 4 + int64_t(sizeof(Unit))) + 16;
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
    if (a.p.tokens_q == 0 || (a.p.batch == 0 && a.p.clear_tail == 0)) return STA_OK;
    auto bad = [](const void* x) { return x == nullptr || reinterpret_cast<uintptr_t>(x) % 4 != 0; };
    if (bad(lse) || (a.p.batch > 0 && (bad(lengths) || bad(block_tables)))) return STA_ERR_INVALID_ARG;
    if (!rows_ok(q, a.p.tokens_q) || !rows_ok(o, a.p.tokens_q)) return STA_ERR_INVALID_ARG;
    int64_t need = 0;
    if (sta_status st = sta_cache_workspace(c, p, &need); st != STA_OK) return st;
    if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || workspace_bytes < need)
        return STA_ERR_INVALID_ARG;
    if (cudaError_t e = op_begin(); e != cudaSuccess) return op_cuda_status(e);
    if (cudaError_t e = op_status_word(&a.p.status); e != cudaSuccess) return op_cuda_status(e);
    a.blocks = c->blocks;
    a.bt = c->block_tokens;
    a.bt_log2 = a.bt == 16 ? 4 : a.bt == 32 ? 5 : a.bt == 64 ? 6 : 7;
    a.k_scales = c->k_scales;
    a.v_scales = c->v_scales;
    a.warp_parts = static_cast<float*>(workspace);
    a.timeout_ns = a.p.waits.timeout_ns;
    a.lengths = lengths;
    a.tables = block_tables;
    a.width = table_width;
    a.stride = table_stride;
    a.q = rows_of(q);
    a.o = rows_of(o);
    a.lse = lse;
    int sms = 0;
    if (cudaError_t e = packed::sm_count(&sms); e != cudaSuccess) return op_cuda_status(e);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return op_cuda_status(c->head_dim == 128 ? launch_attention<128>(*c, a, sms, s) : launch_attention<64>(*c, a, sms, s));
}

}  // extern "C"
