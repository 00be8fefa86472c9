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

// One warp streams tiles of 32 tokens through its own ring in shared memory; a CTA is 8
// such warps and has its SM alone (192 KB of ring: 24 KB in flight for each warp, several
// times what 1 us of HBM latency needs).
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;      // tokens of a tile
constexpr int kRowTile = 16;   // query rows of a unit: one mma.m16n8k16 A operand
constexpr int kMaxSms = 148;   // of a B200, for workspaces asked for without a device
constexpr int kMinTiles = 8;   // a CTA takes no fewer tiles than it has warps
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct CacheArgs {
    PackedProblem p;
    int32_t blocks, bt;
    const float* k_scales;
    const float* v_scales;
    const int32_t* lengths;
    const int32_t* tables;
    int32_t width;
    int64_t stride;
    Rows q, o;
    float* lse;
    float* parts;  // [2 * CTAs][16 rows][D + 4]: O, m, l, mw
    uint64_t timeout_ns;
};

// The work: units of (sequence, 16 query rows, key head), each of the sequence's tiles; all
// units' tiles in one row, cut into equal runs, one for each CTA.  A unit that lies in one
// run is finished there; the others' parts are joined by the second kernel, in the
// order of the runs.
struct Sequence {
    int32_t q0, nq;      // its queries
    int32_t len, raw;    // tokens in the table; as given
    int32_t tiles;       // at least 1
    int32_t units;       // row tiles * key heads
};

__device__ __forceinline__ Sequence sequence(const CacheArgs& a, int b, bool* cut) {
    Sequence s;
    s.q0 = b;
    s.nq = 1;
    if (a.p.cu_q != nullptr) {
        const int32_t c0 = a.p.cu_q[b], c1 = a.p.cu_q[b + 1];
        s.q0 = max(0, min(c0, a.p.tokens_q));
        s.nq = max(s.q0, min(c1, a.p.tokens_q)) - s.q0;
        *cut |= c0 != s.q0 || c1 != s.q0 + s.nq;
    }
    s.raw = a.lengths[b];
    s.len = max(0, min(s.raw, a.width * a.bt));
    *cut |= s.raw != s.len;
    s.tiles = max(1, (s.len + kTile - 1) / kTile);
    s.units = (s.nq * a.p.group + kRowTile - 1) / kRowTile * a.p.kv_heads;
    return s;
}

struct PlanShared {
    int64_t scan[kWarps];
    int64_t total;
    int64_t before;   // tiles of the sequences before `seq`
    int32_t seq;
    int32_t last;     // end of the last sequence's queries
};

// Tiles of all units; the last query row.
__device__ int64_t plan_total(const CacheArgs& a, PlanShared& sh, bool report) {
    int64_t n = 0;
    int32_t last = 0;
    bool cut = false;
    for (int b = threadIdx.x; b < a.p.batch; b += kThreads) {
        const Sequence s = sequence(a, b, &cut);
        n += int64_t(s.tiles) * s.units;
        last = max(last, s.q0 + s.nq);
    }
    for (int i = 16; i > 0; i >>= 1) {
        n += __shfl_xor_sync(~0u, n, i);
        last = max(last, __shfl_xor_sync(~0u, last, i));
    }
    if (threadIdx.x == 0) sh.last = 0;
    __syncthreads();
    if (threadIdx.x % 32 == 0) {
        sh.scan[threadIdx.x / 32] = n;
        atomicMax(&sh.last, last);
    }
    if (__syncthreads_or(cut) && report && threadIdx.x == 0) atomicOr(a.p.status, kDevBounds);
    n = 0;
    for (int i = 0; i < kWarps; ++i) n += sh.scan[i];
    __syncthreads();
    return n;
}

// The sequence that holds tile `at` (sh.seq) and the tiles before it (sh.before).
__device__ void plan_locate(const CacheArgs& a, PlanShared& sh, int64_t at) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t carry = 0;
    if (threadIdx.x == 0) sh.seq = -1;
    __syncthreads();
    for (int b0 = 0; b0 < a.p.batch; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        bool cut = false;
        int64_t v = 0;
        if (b < a.p.batch) {
            const Sequence s = sequence(a, b, &cut);
            v = int64_t(s.tiles) * s.units;
        }
        int64_t x = v;
        for (int i = 1; i < 32; i <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, x, i);
            if (lane >= i) x += y;
        }
        if (lane == 31) sh.scan[warp] = x;
        __syncthreads();
        int64_t base = carry;
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) base += sh.scan[i];
            carry += sh.scan[i];
        }
        if (v > 0 && at >= base + x - v && at < base + x) {
            sh.seq = b;
            sh.before = base + x - v;
        }
        __syncthreads();
        if (carry > at) break;
    }
}

// CTAs that take part, and the first tile of CTA i of them.
__device__ __forceinline__ int64_t plan_ctas(int64_t total, int64_t grid) {
    const int64_t most = (total + kMinTiles - 1) / kMinTiles;
    return most < grid ? most : grid;
}
__device__ __forceinline__ int64_t plan_first(int64_t total, int64_t ctas, int64_t i) {
    return total / ctas * i + total % ctas * i / ctas;
}

// D += A B, m16n8k16, fp16 operands, fp32 accumulators.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
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
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Writes one row's D / 16 outputs from `col` on, and its LSE.
template <int D>
__device__ __forceinline__ void store_row(const CacheArgs& a, int32_t tok, int32_t head, int col, const float* x, float m,
                                          float l, float mw) {
    constexpr int E = D / 16;
    const bool none = l == 0.0f;
    const float f = none ? 0.0f : ptx::ex2(mw - m) / l;
    __nv_bfloat16* dst = a.o.p + int64_t(tok) * a.o.ts + head * a.o.hs + col;
    uint32_t pk[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) pk[i] = none ? 0u : ptx::pack_bf16x2(x[2 * i] * f, x[2 * i + 1] * f);
    if (E == 8)
        *reinterpret_cast<uint4*>(dst) = make_uint4(pk[0], pk[1], pk[E / 2 - 2], pk[E / 2 - 1]);
    else
        *reinterpret_cast<uint2*>(dst) = make_uint2(pk[0], pk[1]);
    if (col == 0) a.lse[int64_t(head) * a.p.tokens_q + tok] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Attention over the cache.  For each tile a warp holds S (16 x 32) and O (16 x D) in registers:
// S = Q K^T, P = 2^(S - m), O += W V by mma.m16n8k16 on fp16 operands with fp32 sums; the codes
// become fp16 exactly (cvt), so no tensor is widened in memory.  Both products pick their
// operands' order freely over the summed index: K's 16 bytes of a thread are four k-steps, V's
// 16 bytes of two tokens sixteen output columns, and neither is ever transposed.
// A block's K scale multiplies the scores.  Its V scale 2^lv enters the exponent: W = 2^(S + lv - mw)
// with a running maximum mw of its own, so that W rounds to fp16 (2^-11 relative) relative to
// each row's largest contribution, however far the scales are apart; l sums the unscaled P
// before any rounding.  Q is scaled by a power of two for each row into fp16's range.
// HBM-bound: 2 D bytes for each token and key head; mma.sync suffices (a few rows of queries
// leave a 128-row tcgen05 tile mostly empty, and the codes would have to be widened in
// shared memory first).
template <int D>
struct Cfg {
    static constexpr int kTileBytes = kTile * D;           // of K or V
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kRing = kWarps * kStages * 2 * kTileBytes;
    static constexpr int kMetaOff = kRing;                 // {ks0, ks1, lv0, lv1} for each warp and stage
    static constexpr int kBarOff = kMetaOff + kWarps * kStages * 16;
    static constexpr int kStatOff = kBarOff + kWarps * kStages * 8;  // [3][8 warps][16 rows]: m, l, mw
    static constexpr int kSmem = kStatOff + 3 * kWarps * kRowTile * 4 + 1024;
    static_assert(kWarps * kRowTile * (D + 4) * 4 <= kRing, "the warps' O fit in the ring");
    static_assert(kSmem <= 226 * 1024, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cache_attention_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const CacheArgs a) {
    using C = Cfg<D>;
    constexpr int S = C::kStages;
    constexpr int kSteps = D / 16;    // k-steps of Q K^T
    constexpr int kCols = D / 8;      // 8-column tiles of O
    extern __shared__ uint8_t smem_raw[];
    __shared__ PlanShared plan;
    const uint32_t raw_base = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int K = a.p.kv_heads, G = a.p.group;
    float4* meta = reinterpret_cast<float4*>(smem + C::kMetaOff) + warp * S;
    const uint32_t bar0 = base + C::kBarOff + warp * S * 8;
    uint8_t* ring = smem + warp * S * 2 * C::kTileBytes;
    float* part_o = reinterpret_cast<float*>(smem);       // [8 warps][16 rows][D + 4], over the rings
    float* stat = reinterpret_cast<float*>(smem + C::kStatOff);
    if (lane == 0) {
        for (int i = 0; i < S; ++i) ptx::mbar_init(bar0 + 8u * i, 1);
        ptx::fence_barrier_init();
    }
    __syncwarp();
    ops::grid_launch_dependents();

    const int64_t total = plan_total(a, plan, blockIdx.x == 0);
    if (a.p.clear_tail && plan.last < a.p.tokens_q) {
        const int32_t tail = a.p.tokens_q - plan.last, parts = D / 8;
        for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < int64_t(tail) * a.p.heads * parts;
             i += int64_t(gridDim.x) * kThreads) {
            const int64_t row = i / parts;
            const int32_t tok = plan.last + int32_t(row / a.p.heads), h = int32_t(row % a.p.heads);
            *reinterpret_cast<uint4*>(a.o.p + tok * a.o.ts + h * a.o.hs + i % parts * 8) = make_uint4(0u, 0u, 0u, 0u);
            if (i % parts == 0) a.lse[int64_t(h) * a.p.tokens_q + tok] = -INFINITY;
        }
    }
    const int64_t ctas = plan_ctas(total, gridDim.x);
    if (blockIdx.x >= ctas) return;
    int64_t at = plan_first(total, ctas, blockIdx.x);
    const int64_t end = plan_first(total, ctas, blockIdx.x + 1);
    plan_locate(a, plan, at);
    int32_t b = plan.seq;
    int64_t before = plan.before;
    uint32_t issued = 0, taken = 0;  // tiles of this warp so far: ring slot and phase
    bool dead = false;

    while (at < end) {
        bool cut = false;
        const Sequence sq = sequence(a, b, &cut);
        const int64_t in_seq = at - before;
        if (in_seq >= int64_t(sq.tiles) * sq.units) {
            before += int64_t(sq.tiles) * sq.units;
            ++b;
            continue;
        }
        const int unit = int(in_seq / sq.tiles), first = int(in_seq % sq.tiles);
        const int rt = unit / K, hk = unit % K;
        const int last = int(min(int64_t(sq.tiles), first + (end - at)));
        at += last - first;
        // ---- this warp's tiles
        const int n = last - first;
        const int t0 = first + n * warp / kWarps, t1 = first + n * (warp + 1) / kWarps;
        const int rows = min(kRowTile, sq.nq * G - rt * kRowTile);
        // keys that row r sees: the first raw - nq + token + 1; never more than the table holds
        auto limit_of = [&](int r) { return min(sq.len, sq.raw - sq.nq + (rt * kRowTile + r) / G + 1); };
        const int limit_a = g < rows ? limit_of(g) : INT32_MAX, limit_b = g + 8 < rows ? limit_of(g + 8) : INT32_MAX;
        const int least = limit_of(0);  // the smallest limit of the rows

        // ---- pages: lane i holds page `p0 + i` of the warp's run
        const int bt = a.bt, pages = (sq.len + bt - 1) / bt;
        const int32_t* table = a.tables + int64_t(b) * a.stride;
        int p0 = -1, page_id = 0;
        float page_ks = 0.0f, page_lv = 0.0f;  // ks < 0: not to be seen
        auto load_pages = [&](int from) {
            p0 = from;
            const int j = from + lane;
            int id = j < pages ? table[j] : 0;
            const bool bad = id < 0 || id >= a.blocks;
            if (bad) {
                atomicOr(a.p.status, kDevBounds);
                id = 0;
            }
            page_id = id;
            page_ks = j < pages && !bad ? a.k_scales[int64_t(id) * K + hk] : -1.0f;
            page_lv = j < pages && !bad ? log2f(a.v_scales[int64_t(id) * K + hk]) : 0.0f;
        };
        auto issue = [&](int tile) {
            const int tok = tile * kTile, pg = tok / bt;
            if (p0 < 0 || pg >= p0 + 32 || (bt < kTile && pg + 1 >= p0 + 32)) load_pages(pg);
            const int id0 = __shfl_sync(~0u, page_id, pg - p0), id1 = __shfl_sync(~0u, page_id, (pg - p0 + 1) & 31);
            float4 mt;
            mt.x = __shfl_sync(~0u, page_ks, pg - p0);
            mt.z = __shfl_sync(~0u, page_lv, pg - p0);
            mt.y = __shfl_sync(~0u, page_ks, (pg - p0 + 1) & 31);
            mt.w = __shfl_sync(~0u, page_lv, (pg - p0 + 1) & 31);
            const int slot = int(issued % S);
            if (lane == 0) {
                if (bt >= kTile) {
                    mt.y = mt.x;
                    mt.w = mt.z;
                }
                meta[slot] = mt;
                const uint32_t bar = bar0 + 8u * slot, dst = ptx::smem_u32(ring + slot * 2 * C::kTileBytes);
                ptx::mbar_arrive_expect_tx(bar, 2 * C::kTileBytes);
                const int32_t r0 = (id0 * K + hk) * bt + tok % bt;
                ptx::tma_load_2d(dst, &tm_k, bar, 0, r0);
                ptx::tma_load_2d(dst + C::kTileBytes, &tm_v, bar, 0, r0);
                if (bt < kTile) {
                    const int32_t r1 = (id1 * K + hk) * bt;
                    ptx::tma_load_2d(dst + C::kTileBytes / 2, &tm_k, bar, 0, r1);
                    ptx::tma_load_2d(dst + C::kTileBytes + C::kTileBytes / 2, &tm_v, bar, 0, r1);
                }
            }
            ++issued;
        };
        int next = t0;
        for (; next < t1 && next < t0 + S; ++next) issue(next);

        // ---- Q as the A operand of every k-step: thread (g, t) holds 16-element pieces t, t + 4 of rows g, g + 8
        uint32_t qa[kSteps][4];
        float rf_a, rf_b;  // scores of the two rows: factor of the products
        {
            uint32_t raw[2][D / 8];  // [row][pairs]
            float top[2] = {0.0f, 0.0f};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = rt * kRowTile + g + 8 * r;
                const bool have = g + 8 * r < rows;
                const __nv_bfloat16* src =
                    a.q.p + int64_t(sq.q0 + (have ? row / G : 0)) * a.q.ts + (hk * G + (have ? row % G : 0)) * a.q.hs;
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        uint4 u = make_uint4(0u, 0u, 0u, 0u);
                        if (have) u = __ldg(reinterpret_cast<const uint4*>(src + (t + 4 * c) * 16 + hh * 8));
                        raw[r][c * 8 + hh * 4 + 0] = u.x;
                        raw[r][c * 8 + hh * 4 + 1] = u.y;
                        raw[r][c * 8 + hh * 4 + 2] = u.z;
                        raw[r][c * 8 + hh * 4 + 3] = u.w;
                    }
#pragma unroll
                for (int i = 0; i < D / 8; ++i) top[r] = fmaxf(top[r], fmaxf(fabsf(bf_lo(raw[r][i])), fabsf(bf_hi(raw[r][i]))));
                top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 2));
            }
            float sc[2], rf[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                // 2^e with |q| 2^e < 512: fp16 keeps elements down to 2^-33 of the largest
                const int e = min(max(8 - (int(__float_as_uint(top[r]) >> 23) - 126), -119), 126);
                sc[r] = __uint_as_float(uint32_t(e + 127) << 23);
                rf[r] = a.p.scale * kLog2e * __uint_as_float(uint32_t(127 - e) << 23);
            }
            rf_a = rf[0];
            rf_b = rf[1];
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t u0 = raw[r][c * 8 + 2 * s], u1 = raw[r][c * 8 + 2 * s + 1];
                        qa[c * 4 + s][r] = half2_of(bf_lo(u0) * sc[r], bf_hi(u0) * sc[r]);
                        qa[c * 4 + s][2 + r] = half2_of(bf_lo(u1) * sc[r], bf_hi(u1) * sc[r]);
                    }
        }

        float o[kCols][4];
#pragma unroll
        for (int j = 0; j < kCols; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
        float m_a = -INFINITY, m_b = -INFINITY, w_a = -INFINITY, w_b = -INFINITY, l_a = 0.0f, l_b = 0.0f;

        for (int tile = t0; tile < t1; ++tile) {
            const int slot = int(taken % S);
            const uint32_t bar = bar0 + 8u * slot, phase = (taken / S) & 1u;
            if (!__all_sync(~0u, ptx::mbar_try_wait(bar, phase))) {
                const uint64_t from = ptx::globaltimer_ns();
                while (!ptx::mbar_try_wait(bar, phase))
                    if (ptx::globaltimer_ns() - from > a.timeout_ns) {
                        dead = true;  // give up waiting; the results are lost and reported
                        if (lane == 0) atomicOr(a.p.status, kDevTimeout);
                        break;
                    }
                if (__any_sync(~0u, dead)) {  // the warp stops together, and issues no more
                    dead = true;
                    break;
                }
            }
            const float4 mt = meta[slot];
            const uint8_t* kt = ring + slot * 2 * C::kTileBytes;
            const uint8_t* vt = kt + C::kTileBytes;
            // ---- S = Q K^T: four 8-token tiles
            float s[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
                const int row = i * 8 + g;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const int chunk = t + 4 * c;
                    const int off = D == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4) : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
                    const uint4 u = *reinterpret_cast<const uint4*>(kt + off);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mma16816(s[i], qa[c * 4 + q], ops::e4m3_half2(uint16_t(w[q])), ops::e4m3_half2(uint16_t(w[q] >> 16)));
                }
            }
            // ---- scores in units of log2; masks
            const int tok = tile * kTile;
            const bool masked = tok + kTile > least || mt.x < 0.0f || mt.y < 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float ks = i < 2 ? mt.x : mt.y;
                s[i][0] *= rf_a * ks;
                s[i][1] *= rf_a * ks;
                s[i][2] *= rf_b * ks;
                s[i][3] *= rf_b * ks;
                if (masked) {
                    const int j = tok + i * 8 + 2 * t;
                    const bool out = ks < 0.0f;
                    if (out || j >= limit_a) s[i][0] = -INFINITY;
                    if (out || j + 1 >= limit_a) s[i][1] = -INFINITY;
                    if (out || j >= limit_b) s[i][2] = -INFINITY;
                    if (out || j + 1 >= limit_b) s[i][3] = -INFINITY;
                }
            }
            float xa0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
            float xa1 = fmaxf(fmaxf(s[2][0], s[2][1]), fmaxf(s[3][0], s[3][1]));
            float xb0 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
            float xb1 = fmaxf(fmaxf(s[2][2], s[2][3]), fmaxf(s[3][2], s[3][3]));
#pragma unroll
            for (int i = 1; i <= 2; i <<= 1) {
                xa0 = fmaxf(xa0, __shfl_xor_sync(~0u, xa0, i));
                xa1 = fmaxf(xa1, __shfl_xor_sync(~0u, xa1, i));
                xb0 = fmaxf(xb0, __shfl_xor_sync(~0u, xb0, i));
                xb1 = fmaxf(xb1, __shfl_xor_sync(~0u, xb1, i));
            }
            const float mn_a = fmaxf(m_a, fmaxf(xa0, xa1)), mn_b = fmaxf(m_b, fmaxf(xb0, xb1));
            const float wn_a = fmaxf(w_a, fmaxf(xa0 + mt.z, xa1 + mt.w)), wn_b = fmaxf(w_b, fmaxf(xb0 + mt.z, xb1 + mt.w));
            const float mu_a = mn_a == -INFINITY ? 0.0f : mn_a, mu_b = mn_b == -INFINITY ? 0.0f : mn_b;
            const float wu_a = wn_a == -INFINITY ? 0.0f : wn_a, wu_b = wn_b == -INFINITY ? 0.0f : wn_b;
            if (__any_sync(~0u, mn_a != m_a || mn_b != m_b || wn_a != w_a || wn_b != w_b)) {
                l_a *= ptx::ex2(m_a - mu_a);
                l_b *= ptx::ex2(m_b - mu_b);
                const float ca = ptx::ex2(w_a - wu_a), cb = ptx::ex2(w_b - wu_b);
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    o[j][0] *= ca;
                    o[j][1] *= ca;
                    o[j][2] *= cb;
                    o[j][3] *= cb;
                }
                m_a = mn_a;
                m_b = mn_b;
                w_a = wn_a;
                w_b = wn_b;
            }
            // W = P 2^(m + lv - mw); where that factor is past fp32, P is 0
            const float fa[2] = {ptx::ex2(fminf(mu_a + mt.z - wu_a, 126.0f)), ptx::ex2(fminf(mu_a + mt.w - wu_a, 126.0f))};
            const float fb[2] = {ptx::ex2(fminf(mu_b + mt.z - wu_b, 126.0f)), ptx::ex2(fminf(mu_b + mt.w - wu_b, 126.0f))};
            uint32_t pa[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p0_ = ptx::ex2(s[i][0] - mu_a), p1_ = ptx::ex2(s[i][1] - mu_a);
                const float p2_ = ptx::ex2(s[i][2] - mu_b), p3_ = ptx::ex2(s[i][3] - mu_b);
                l_a += p0_ + p1_;
                l_b += p2_ + p3_;
                pa[i / 2][(i & 1) * 2] = half2_of(p0_ * fa[i / 2], p1_ * fa[i / 2]);
                pa[i / 2][(i & 1) * 2 + 1] = half2_of(p2_ * fb[i / 2], p3_ * fb[i / 2]);
            }
            // ---- O += W V: two 16-token steps; thread (g, t) takes tokens 2t, 2t + 1, 2t + 8, 2t + 9
            // and D / 8 columns from g * D / 8 on
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t v[4][D / 32];  // [token][words]
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = q * 16 + 2 * t + (i & 1) + (i >> 1) * 8;
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
                    if (masked && (tok + row >= sq.len || (q == 0 ? mt.x : mt.y) < 0.0f))
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) v[i][j] = 0u;
                }
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const uint32_t a0 = __byte_perm(v[0][j], v[1][j], 0x5140), a1 = __byte_perm(v[0][j], v[1][j], 0x7362);
                    const uint32_t c0 = __byte_perm(v[2][j], v[3][j], 0x5140), c1 = __byte_perm(v[2][j], v[3][j], 0x7362);
                    mma16816(o[4 * j + 0], pa[q], ops::e4m3_half2(uint16_t(a0)), ops::e4m3_half2(uint16_t(c0)));
                    mma16816(o[4 * j + 1], pa[q], ops::e4m3_half2(uint16_t(a0 >> 16)), ops::e4m3_half2(uint16_t(c0 >> 16)));
                    mma16816(o[4 * j + 2], pa[q], ops::e4m3_half2(uint16_t(a1)), ops::e4m3_half2(uint16_t(c1)));
                    mma16816(o[4 * j + 3], pa[q], ops::e4m3_half2(uint16_t(a1 >> 16)), ops::e4m3_half2(uint16_t(c1 >> 16)));
                }
            }
            ++taken;
            __syncwarp();  // every lane has read the slot
            if (next < t1) issue(next++);
        }
        l_a += __shfl_xor_sync(~0u, l_a, 1);
        l_a += __shfl_xor_sync(~0u, l_a, 2);
        l_b += __shfl_xor_sync(~0u, l_b, 1);
        l_b += __shfl_xor_sync(~0u, l_b, 2);

        // ---- join the warps: O over the rings (every copy has been taken), columns of row r at 32 t ..
        __syncthreads();
        {
            float* dst = part_o + (warp * kRowTile + g) * (D + 4);
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                // column tile j: n = 2t, 2t + 1 are columns 2t * D/8 + j and (2t + 1) * D/8 + j
                dst[2 * t * (D / 8) + j] = o[j][0];
                dst[(2 * t + 1) * (D / 8) + j] = o[j][1];
                dst[8 * (D + 4) + 2 * t * (D / 8) + j] = o[j][2];
                dst[8 * (D + 4) + (2 * t + 1) * (D / 8) + j] = o[j][3];
            }
            if (t == 0) {
                float* st = stat + warp * kRowTile + g;
                st[0] = m_a;
                st[8] = m_b;
                st[kWarps * kRowTile] = l_a;
                st[kWarps * kRowTile + 8] = l_b;
                st[2 * kWarps * kRowTile] = w_a;
                st[2 * kWarps * kRowTile + 8] = w_b;
            }
        }
        __syncthreads();
        {
            constexpr int E = D / 16;
            const int row = threadIdx.x / 16, col = (threadIdx.x % 16) * E;
            float m = -INFINITY, mw = -INFINITY, l = 0.0f, x[E];
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = 0.0f;
            for (int w = 0; w < kWarps; ++w) {
                m = fmaxf(m, stat[w * kRowTile + row]);
                mw = fmaxf(mw, stat[(2 * kWarps + w) * kRowTile + row]);
            }
            const float mu = m == -INFINITY ? 0.0f : m, wu = mw == -INFINITY ? 0.0f : mw;
            for (int w = 0; w < kWarps; ++w) {
                const float f = ptx::ex2(stat[(2 * kWarps + w) * kRowTile + row] - wu);
                l += stat[(kWarps + w) * kRowTile + row] * ptx::ex2(stat[w * kRowTile + row] - mu);
                const float* src = part_o + (w * kRowTile + row) * (D + 4) + col;
#pragma unroll
                for (int i = 0; i < E; ++i) x[i] += src[i] * f;
            }
            if (first == 0 && last == sq.tiles) {
                const int r = rt * kRowTile + row;
                if (row < rows) store_row<D>(a, sq.q0 + r / G, hk * G + r % G, col, x, mu, l, wu);
            } else {
                // a part of the unit: a run that began in an earlier CTA is this CTA's first
                const int64_t slot = 2 * int64_t(blockIdx.x) + (first > 0 ? 0 : 1);
                float* dst = a.parts + (slot * kRowTile + row) * (D + 4);
#pragma unroll
                for (int i = 0; i < E; ++i) dst[col + i] = x[i];
                if (col == 0) {
                    dst[D] = m;
                    dst[D + 1] = l;
                    dst[D + 2] = mw;
                }
            }
        }
        ptx::fence_proxy_async_smem();  // the rings are written by copies again
        __syncthreads();
        if (__syncthreads_or(dead)) break;
    }
    // After a wait that ran out: the copies still in flight land before the CTA leaves (bounded).
    if (dead)
        for (; taken < issued; ++taken) drain_bar(bar0 + 8u * (taken % S), (taken / S) & 1u, a.timeout_ns);
}

// Joins the parts of the units that lie in several CTAs' runs: CTA i takes the unit that
// its run begins inside of, if that is the unit's first such run.
template <int D>
__global__ void __launch_bounds__(kThreads) cache_join_kernel(const CacheArgs a, int grid) {
    __shared__ PlanShared plan;
    ops::grid_wait();
    const int64_t total = plan_total(a, plan, false), ctas = plan_ctas(total, grid);
    const int64_t i = int64_t(blockIdx.x) + 1;
    if (i >= ctas) return;
    const int64_t at = plan_first(total, ctas, i);
    plan_locate(a, plan, at);
    bool cut = false;
    const Sequence sq = sequence(a, plan.seq, &cut);
    const int unit = int((at - plan.before) / sq.tiles);
    const int64_t unit0 = plan.before + int64_t(unit) * sq.tiles, unit1 = unit0 + sq.tiles;
    if (at == unit0 || plan_first(total, ctas, i - 1) > unit0) return;
    constexpr int E = D / 16;
    const int row = threadIdx.x / 16, col = (threadIdx.x % 16) * E;
    const int K = a.p.kv_heads, G = a.p.group, rt = unit / K, hk = unit % K, r = rt * kRowTile + row;
    if (r >= sq.nq * G) return;
    const float* first = a.parts + ((2 * (i - 1) + 1) * kRowTile + row) * (D + 4);
    float m = first[D], mw = first[D + 2];
    int64_t parts = 0;
    for (int64_t c = i; c < ctas && plan_first(total, ctas, c) < unit1; ++c, ++parts) {
        const float* p = a.parts + (2 * c * kRowTile + row) * (D + 4);
        m = fmaxf(m, p[D]);
        mw = fmaxf(mw, p[D + 2]);
    }
    const float mu = m == -INFINITY ? 0.0f : m, wu = mw == -INFINITY ? 0.0f : mw;
    float l = first[D + 1] * ptx::ex2(first[D] - mu), x[E];
    float f = ptx::ex2(first[D + 2] - wu);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = first[col + e] * f;
    for (int64_t c = i; c < i + parts; ++c) {
        const float* p = a.parts + (2 * c * kRowTile + row) * (D + 4);
        l += p[D + 1] * ptx::ex2(p[D] - mu);
        f = ptx::ex2(p[D + 2] - wu);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] += p[col + e] * f;
    }
    store_row<D>(a, sq.q0 + r / G, hk * G + r % G, col, x, mu, l, wu);
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

template <int D>
cudaError_t launch_attention(const sta_cache& c, const CacheArgs& a, int sms, cudaStream_t stream) {
    const int64_t n_rows = int64_t(c.blocks) * c.kv_heads * c.block_tokens;
    const int box = c.block_tokens < kTile ? c.block_tokens : kTile;
    CUtensorMap mk, mv;
    cudaError_t e = codes_map(&mk, c.k_codes, n_rows, D, box);
    if (e == cudaSuccess) e = codes_map(&mv, c.v_codes, n_rows, D, box);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(cache_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e == cudaSuccess)
        e = packed::launch(cache_attention_kernel<D>, unsigned(sms), kThreads, Cfg<D>::kSmem, stream, false, mk, mv, a);
    if (e == cudaSuccess && sms > 1)
        e = packed::launch(cache_join_kernel<D>, unsigned(sms - 1), kThreads, 0, stream, true, a, sms);
    return e;
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
    int sms = 0;
    if (packed::sm_count(&sms) != cudaSuccess) {
        (void)cudaGetLastError();
        sms = kMaxSms;  // no device here: as for the largest
    }
    *bytes = int64_t(2) * sms * kRowTile * (c->head_dim + 4) * 4;
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
    a.blocks = c->blocks;
    a.bt = c->block_tokens;
    a.k_scales = c->k_scales;
    a.v_scales = c->v_scales;
    a.parts = static_cast<float*>(workspace);
    a.timeout_ns = kOpTimeoutNs;
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
