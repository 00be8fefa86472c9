// sta_packed.cuh -- the work lists of the packed attention, built on the device
// from the sequences' bounds, and the tensor maps of token-major tensors.
//
// Rows.  A query block is up to 128 rows of one sequence and one key head: the
// G = heads / kv_heads query heads that share the key head stand side by side,
// row r = token r / G, head r % G, so a block covers T = 128 / G tokens.  Rows of
// short sequences then fill a block G times better than one head's would, the
// causal diagonal wastes T tokens of a key chunk instead of 128, and the
// gradients of a shared key head are sums over one block's rows.  A key block is
// 128 keys of one sequence and key head.  The lists hold blocks, ordered by
// falling work; an item is (block, key head).
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
    int32_t pad[2];
};
struct alignas(16) KBlock {
    int32_t key0, nkeys;    // first key (row of the tensors), keys (1..128)
    int32_t pos;            // its position in the sequence
    int32_t q0, nq;         // the query blocks that see it: [q0, q0 + nq)
    int32_t pad[3];
};

// Head of the workspace.
struct Lists {
    int32_t n_q, n_k;       // blocks
    int32_t next_q, next_k, next_dq;  // item counters of the kernels (zeroed with the lists)
};

// Offsets into the workspace, from the problem's sizes alone.
struct Layout {
    int64_t qblocks, kblocks, order_q, order_k, bounds, neg_l, neg_d, bytes;
    int64_t max_q, max_k;
};

inline int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

inline Layout layout(const PackedProblem& p, bool backward) {
    Layout w{};
    const int tpb = kRows / p.group;
    w.max_q = p.tokens_q / tpb + p.batch;
    w.max_k = backward ? p.tokens_k / kRows + p.batch : 0;
    int64_t at = 256;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up256(bytes);
        return here;
    };
    w.qblocks = take(w.max_q * sizeof(QBlock));
    w.kblocks = take(w.max_k * sizeof(KBlock));
    w.order_q = take(w.max_q * 4);
    w.order_k = take(w.max_k * 4);
    w.bounds = take((int64_t(p.batch) + 1) * 4 * 4);
    if (backward) {
        w.neg_l = take(w.max_q * p.kv_heads * kRows * 4);
        w.neg_d = take(w.max_q * p.kv_heads * kRows * 4);
    }
    w.bytes = at;
    return w;
}

// Device view of the lists.
struct View {
    Lists* lists;
    QBlock* qblocks;
    KBlock* kblocks;
    int32_t* order_q;
    int32_t* order_k;
    int32_t* bounds;  // [4][batch + 1]: cut cu_q, cut cu_k, first query block, first key block
};
inline View view(const Layout& w, void* ws) {
    char* b = static_cast<char*>(ws);
    return View{reinterpret_cast<Lists*>(b), reinterpret_cast<QBlock*>(b + w.qblocks),
                reinterpret_cast<KBlock*>(b + w.kblocks), reinterpret_cast<int32_t*>(b + w.order_q),
                reinterpret_cast<int32_t*>(b + w.order_k), reinterpret_cast<int32_t*>(b + w.bounds)};
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

// Launch attributes: `pdl`: the kernel may start while its predecessor in the
// stream ends, and waits for it (griddepcontrol.wait) before it reads memory.
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, bool pdl,
                   A&&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
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

}  // namespace packed
}  // namespace sta
