// sta_packed.cuh -- the work lists of the packed attention, built on the device
// from the sequences' bounds, and the tensor maps of token-major tensors.
//
// Rows.  A query block is up to 128 rows of one sequence and one key head: the
// G = heads / kv_heads query heads that share the key head stand side by side,
// row r = token r / G, head r % G, so a block covers T = 128 / G tokens.  Rows of
// short sequences then fill a block G times better than one head's would, the
// causal diagonal wastes T tokens of a key chunk instead of 128, and the
// gradients of a shared key head are sums over one block's rows.  A key block is
// 128 keys of one sequence and key head.
//
// Work.  A query block walks the 128-key chunks that it sees, a key block the query
// blocks that see it.  Where there are too few blocks to level the GPU (the caller's
// rule on sizes), long walks are split into parts: each part keeps fp32 sums in the
// workspace, a last kernel joins them in order.  The lists hold the walks (whole or
// parts), longest first; an item is (walk, key head).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sta_ops.h"

namespace sta {
namespace packed {

constexpr int kRows = 128;  // rows of a query block, keys of a key block or chunk

struct alignas(16) QBlock {
    int32_t tok0, ntok;     // first token (row of the tensors), tokens
    int32_t key0, nkeys;    // the sequence's keys
    int32_t limit0;         // keys that the block's first token sees (< 1: none); causal: one more for each token
    int32_t chunks;         // 128-key chunks to walk, at least 1
    int32_t split;          // parts of its walk (1: whole)
    int32_t slot;           // split: first of the parts' places in the workspace
};
struct alignas(16) KBlock {
    int32_t key0, nkeys;    // first key (row of the tensors), keys (1..128)
    int32_t pos;            // its position in the sequence
    int32_t q0, nq;         // the query blocks that see it: [q0, q0 + nq)
    int32_t split, slot;    // as above
    int32_t pad;
};
// A walk, or a part of one, as the kernels' load warps take it (n < 0: no more).
struct alignas(16) QWork {
    int32_t tok0, ntok, key0, nkeys;
    int32_t limit0, c0, n, slot;   // chunks [c0, c0 + n); slot < 0: whole
    int32_t block, hk, pad[2];     // query block; key head (set by the load warp)
};
struct alignas(16) KWork {
    int32_t key0, nkeys, pos, q0;
    int32_t n, slot, hk, pad;      // query blocks [q0, q0 + n)
};

// Head of the workspace.
struct Lists {
    int32_t n_q, n_k;                 // blocks
    int32_t w_q, w_k;                 // walks
    int32_t next_q, next_k, next_dq;  // item counters of the kernels (zeroed with the lists)
};

constexpr int kSplitParts = 4;  // split walks have at most this many parts to an SM, over all key heads
constexpr int kMinPart = 4;     // steps of a part
constexpr int kSplitFrom = 16;  // mean steps of a sequence's longest walk from which splitting is considered

// Offsets into the workspace, from the problem's sizes alone.
struct Layout {
    int64_t qblocks, kblocks, qwalks, kwalks, scratch, bounds, neg_l, neg_d, parts, bytes;
    int64_t max_q, max_k;      // blocks
    int64_t max_wq, max_wk;    // walks
    int32_t split_q, split_k;  // may walks be split?
    int32_t sms;
};

inline int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

// Split where every SM would get fewer than two blocks: with more, the longest walks first
// level the SMs nearly by themselves (a long sequence has many blocks), and the parts' sums
// cost what they save.  (Six sequences of 342-2047 tokens, 16 / 2 heads, d = 64: dK / dV
// 227 us whole, 66 split, plus 10 for the sums; one of 8192 tokens, 24 / 8 heads, d = 128, 520 blocks:
// 730 whole, 848 split.)
inline Layout layout(const PackedProblem& p, bool backward, int head_dim, int sms) {
    Layout w{};
    const int tpb = kRows / p.group;
    w.sms = sms;
    w.max_q = p.tokens_q / tpb + p.batch;
    w.max_k = backward ? p.tokens_k / kRows + p.batch : 0;
    // (nothing to gain where walks are a few steps of a microsecond: the join's launch costs as much)
    const int64_t long_k = int64_t(p.batch) * kSplitFrom * kRows, long_q = int64_t(p.batch) * kSplitFrom * tpb;
    w.split_q = w.max_q * p.kv_heads < 2 * int64_t(sms) && p.tokens_k > long_k;
    w.split_k = backward && w.max_k * p.kv_heads < 2 * int64_t(sms) && p.tokens_q > long_q;
    const int64_t extra = int64_t(kSplitParts) * sms;
    w.max_wq = w.max_q + (w.split_q ? extra : 0);
    w.max_wk = w.max_k + (w.split_k ? extra : 0);
    int64_t at = 256;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up256(bytes);
        return here;
    };
    w.qblocks = take(w.max_q * sizeof(QBlock));
    w.kblocks = take(w.max_k * sizeof(KBlock));
    w.qwalks = take(w.max_wq * sizeof(QWork));
    w.kwalks = take(w.max_wk * sizeof(KWork));
    w.scratch = take((w.max_wq > w.max_wk ? w.max_wq : w.max_wk) * 8);
    w.bounds = take((int64_t(p.batch) + 1) * 4 * 4);
    if (backward) {
        w.neg_l = take(w.max_q * p.kv_heads * kRows * 4);
        w.neg_d = take(w.max_q * p.kv_heads * kRows * 4);
    }
    // parts: O with m and l, or dQ; dK and dV (dQ's are joined before dK / dV's are written)
    const int64_t of_q = w.split_q ? extra * kRows * (head_dim + 2) * 4 : 0;
    const int64_t of_k = w.split_k ? extra * kRows * head_dim * 2 * 4 : 0;
    w.parts = take(of_q > of_k ? of_q : of_k);
    w.bytes = at;
    return w;
}

// Device view of the lists.
struct View {
    Lists* lists;
    QBlock* qblocks;
    KBlock* kblocks;
    QWork* qwalks;
    KWork* kwalks;
    int2* scratch;    // (block, part) of each walk before they are ordered
    int32_t* bounds;  // [4][batch + 1]: cut cu_q, cut cu_k, first query block, first key block
    float* parts;
    int32_t split_q, split_k, sms;
};
inline View view(const Layout& w, void* ws) {
    char* b = static_cast<char*>(ws);
    return View{reinterpret_cast<Lists*>(b), reinterpret_cast<QBlock*>(b + w.qblocks),
                reinterpret_cast<KBlock*>(b + w.kblocks), reinterpret_cast<QWork*>(b + w.qwalks),
                reinterpret_cast<KWork*>(b + w.kwalks), reinterpret_cast<int2*>(b + w.scratch),
                reinterpret_cast<int32_t*>(b + w.bounds), reinterpret_cast<float*>(b + w.parts),
                w.split_q, w.split_k, w.sms};
}

// Rows of outputs to clear behind the last sequence (clear_tail).
struct Tails {
    Rows r[3];
    int32_t heads[3];
    int32_t is_q[3];  // query-like (else key-like)
    int n;
    float* lse;       // or null
};

// One launch: the lists (one CTA) and the tails (the other CTAs, if any).
cudaError_t launch_lists(const PackedProblem& p, const View& v, bool backward, int head_dim, const Tails& tails,
                         cudaStream_t stream);

// Map over a token-major [tokens, heads, d] bf16 tensor: a box is 64 elements x
// `box_heads` heads x `box_tokens` tokens, its rows of 128 bytes in token order
// (heads innermost), 128-byte swizzle.
cudaError_t rows_map(CUtensorMap* m, const Rows& r, int64_t tokens, int heads, int d, int box_heads, int box_tokens);

#ifdef __CUDACC__
// Infinities and NaN where a mask hides them.  In P V a masked pair has P = 0, but 0 x inf and 0 x NaN
// are NaN, and the tensor core multiplies every pair.  So the rows that some row of the block does
// not see have their non-finite elements set to zero in shared memory (scrub_rows), and the rows of
// the result that do see them get them back at the end (restore): adding a non-finite element is
// what its product would have done.  What is scanned is the causal diagonal of a block alone, and
// the second half only runs for an item in which the first found something.
//
// Elements of a pair of bf16 that are not finite: bit 15 for the low one, 31 for the high one.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// Sets those in rows [from, to) of a block in shared memory (128-byte rows in boxes of `box` bytes) to
// zero; `threads` threads share the rows, and the caller fences the writes for the asynchronous proxy.
// Were there any, in the caller's own part?
template <int kBoxes>
__device__ __forceinline__ bool scrub_rows(uint8_t* blk, int box, int from, int to, int thread, int threads) {
    bool any = false;
    for (int i = from * 8 + thread; i < to * 8; i += threads)
#pragma unroll
        for (int cb = 0; cb < kBoxes; ++cb) {
            uint4* at = reinterpret_cast<uint4*>(blk + cb * box + i * 16);
            uint4 x = *at;
            const uint4 b = make_uint4(not_finite(x.x), not_finite(x.y), not_finite(x.z), not_finite(x.w));
            if ((b.x | b.y | b.z | b.w) == 0) continue;
            x.x &= ~((b.x >> 15) * 0xffffu);
            x.y &= ~((b.y >> 15) * 0xffffu);
            x.z &= ~((b.z >> 15) * 0xffffu);
            x.w &= ~((b.w >> 15) * 0xffffu);
            *at = x;
            any = true;
        }
    return any;
}
// r[i] += src[i] where that is not finite, for `n` rows of N elements `stride` apart.
template <int N>
__device__ __forceinline__ void restore(uint32_t (&r)[N], const __nv_bfloat16* src, int64_t stride, int n) {
    for (int k = 0; k < n; ++k) {
        const uint4* row = reinterpret_cast<const uint4*>(src + k * stride);
#pragma unroll
        for (int j = 0; j < N / 8; ++j) {
            const uint4 v = __ldg(row + j);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t b = not_finite(w[e]);
                const int at = 8 * j + 2 * e;
                if (b & 0x8000u) r[at] = __float_as_uint(__uint_as_float(r[at]) + __uint_as_float(w[e] << 16));
                if (b & 0x80000000u)
                    r[at + 1] = __float_as_uint(__uint_as_float(r[at + 1]) + __uint_as_float(w[e] & 0xffff0000u));
            }
        }
    }
}
// Which items had any: word k % kLostWords holds k + 1.  (Writers are at most the item queue's length
// ahead of the last reader, so a word is not reused too early.)
constexpr int kLostWords = 8;
#endif

// Launch attributes: `pdl`: the kernel may start while its predecessor in the stream
// ends, whatever that is, and waits for it (griddepcontrol.wait, in every CTA and before
// any access to global memory, so that its own end says that all before it has ended).
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, bool pdl,
                   A&&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

inline cudaError_t sm_count(int* sms) {
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// The same for workspace sizes, which may be asked for without a device (then a B200's).
inline int sm_count_or_b200() {
    int sms = 0;
    if (sm_count(&sms) == cudaSuccess) return sms;
    (void)cudaGetLastError();
    return 148;
}

}  // namespace packed
}  // namespace sta
