// sta_packed_lists.cu -- the packed attention's work lists (sta_packed.cuh).
#include <cuda_bf16.h>
#include <math.h>

#include <mutex>

#include "sta_ops.cuh"
#include "sta_packed.cuh"

namespace sta {
namespace packed {
namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 1024;     // blocks are ordered by min(work, kBins - 1), falling
constexpr int kNear = 1024;     // up to this many sequences the bounds stay in shared memory

struct Scan {
    int32_t sh[32];
};

// Inclusive scan over the CTA's threads with `op`.
template <class Op>
__device__ int32_t scan(int32_t v, Scan& s, const Op& op) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const int32_t y = __shfl_up_sync(~0u, v, i);
        if (lane >= i) v = op(v, y);
    }
    if (lane == 31) s.sh[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int32_t x = s.sh[lane];
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const int32_t y = __shfl_up_sync(~0u, x, i);
            if (lane >= i) x = op(x, y);
        }
        s.sh[lane] = x;
    }
    __syncthreads();
    if (warp > 0) v = op(v, s.sh[warp - 1]);
    const int32_t r = v;
    __syncthreads();
    return r;
}

// The sequence that block e belongs to: the last b with first[b] <= e.
__device__ int owner(const int32_t* first, int batch, int e) {
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (first[mid] <= e)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Blocks 0 .. n - 1 into `order` by falling work(e); within a bin in any order
// (which block runs first changes no result).
template <class Work>
__device__ void by_work(int32_t n, int32_t* order, int32_t* bins, Scan& s, const Work& work) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) bins[i] = 0;
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += kThreads) atomicAdd(&bins[kBins - 1 - min(work(e), kBins - 1)], 1);
    __syncthreads();
    const int32_t mine = bins[threadIdx.x];
    const int32_t upto = scan(mine, s, [](int32_t a, int32_t b) { return a + b; });
    bins[threadIdx.x] = upto - mine;
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += kThreads)
        order[atomicAdd(&bins[kBins - 1 - min(work(e), kBins - 1)], 1)] = e;
    __syncthreads();
}
static_assert(kBins == kThreads, "one bin for each thread in the scan");

// Zero the rows behind the last sequence (block 0 builds the lists meanwhile).
__device__ void clear_tails(const PackedProblem& p, const Tails& t, int head_dim) {
    // the last bound as block 0 cuts it: the running maximum of the clamped bounds
    __shared__ int32_t last[2];
    if (threadIdx.x < 2) last[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; p.batch > 0 && i <= p.batch; i += blockDim.x) {
        atomicMax(&last[0], min(p.cu_q[i], p.tokens_q));
        atomicMax(&last[1], min(p.cu_k[i], p.tokens_k));
    }
    __syncthreads();
    const int64_t id = int64_t(blockIdx.x - 1) * blockDim.x + threadIdx.x, step = int64_t(gridDim.x - 1) * blockDim.x;
    for (int i = 0; i < t.n; ++i) {
        const int32_t from = t.is_q[i] ? last[0] : last[1], tokens = t.is_q[i] ? p.tokens_q : p.tokens_k;
        const int32_t parts = head_dim / 8;
        const int64_t n = int64_t(tokens - from) * t.heads[i] * parts;
        for (int64_t j = id; j < n; j += step) {
            const int64_t row = j / parts;
            const int32_t tok = from + int32_t(row / t.heads[i]), h = int32_t(row % t.heads[i]);
            *reinterpret_cast<uint4*>(t.r[i].p + tok * t.r[i].ts + h * t.r[i].hs + (j % parts) * 8) =
                make_uint4(0u, 0u, 0u, 0u);
        }
    }
    if (t.lse != nullptr) {
        const int64_t tail = p.tokens_q - last[0];
        for (int64_t j = id; j < tail * p.heads; j += step)
            t.lse[(j / tail) * p.tokens_q + last[0] + j % tail] = -INFINITY;
    }
}

// Latency-bound: a few scans and a counting sort by one CTA; the kernels that
// read the lists start meanwhile and wait.
__global__ void __launch_bounds__(kThreads) packed_lists_kernel(const PackedProblem p, const View v, int backward,
                                                                int head_dim, const Tails tails) {
    ops::grid_launch_dependents();
    if (blockIdx.x > 0) {
        clear_tails(p, tails, head_dim);
        return;
    }
    __shared__ Scan s;
    __shared__ int32_t bins[kBins];
    __shared__ int32_t near_[4][kNear + 1];
    const int B = p.batch, tid = threadIdx.x, tpb = kRows / p.group;
    int32_t* bound[4];  // cut cu_q, cut cu_k, first query block, first key block
    for (int i = 0; i < 4; ++i) bound[i] = B <= kNear ? near_[i] : v.bounds + int64_t(i) * (B + 1);
    const auto max_ = [](int32_t a, int32_t b) { return max(a, b); };
    const auto add_ = [](int32_t a, int32_t b) { return a + b; };
    // ---- bounds cut to the tensors and made rising; blocks counted
    int32_t cq = 0, ck = 0, nbq = 0, nbk = 0;  // carried over passes of 1024 sequences
    bool cut = false;
    if (B > 0) {
        const int32_t a = p.cu_q[0], b = p.cu_k[0];
        cq = max(0, min(a, p.tokens_q));
        ck = max(0, min(b, p.tokens_k));
        cut = a != cq || b != ck;
    }
    if (tid == 0) {
        bound[0][0] = cq;
        bound[1][0] = ck;
        bound[2][0] = bound[3][0] = 0;
    }
    for (int i0 = 0; i0 < B; i0 += kThreads) {
        const int i = i0 + tid;
        const int32_t rq = i < B ? p.cu_q[i + 1] : INT32_MIN, rk = i < B ? p.cu_k[i + 1] : INT32_MIN;
        const int32_t hq = max(cq, scan(min(rq, p.tokens_q), s, max_)), hk = max(ck, scan(min(rk, p.tokens_k), s, max_));
        cut |= i < B && (rq != hq || rk != hk);
        if (i < B) {
            bound[0][i + 1] = hq;
            bound[1][i + 1] = hk;
        }
        __syncthreads();
        const int32_t nq = i < B ? hq - bound[0][i] : 0, nk = i < B ? hk - bound[1][i] : 0;
        const int32_t bq = nbq + scan((nq + tpb - 1) / tpb, s, add_);
        const int32_t bk = backward ? nbk + scan((nk + kRows - 1) / kRows, s, add_) : 0;
        if (i < B) {
            bound[2][i + 1] = bq;
            bound[3][i + 1] = bk;
        }
        __syncthreads();
        const int last = min(i0 + kThreads, B);
        cq = bound[0][last];
        ck = bound[1][last];
        nbq = bound[2][last];
        nbk = bound[3][last];
        __syncthreads();
    }
    if (__syncthreads_or(cut) && tid == 0) atomicOr(p.status, kDevBounds);
    // ---- blocks
    for (int e = tid; e < nbq; e += kThreads) {
        const int b = owner(bound[2], B, e);
        const int32_t q0 = bound[0][b], nq = bound[0][b + 1] - q0, key0 = bound[1][b], nk = bound[1][b + 1] - key0;
        const int32_t t = (e - bound[2][b]) * tpb;
        QBlock q{};
        q.tok0 = q0 + t;
        q.ntok = min(tpb, nq - t);
        q.key0 = key0;
        q.nkeys = nk;
        q.limit0 = p.causal ? nk - nq + t + 1 : nk;
        const int32_t sees = p.causal ? min(nk, q.limit0 + q.ntok - 1) : nk;  // of the block's last token
        q.chunks = max(1, (sees + kRows - 1) / kRows);
        v.qblocks[e] = q;
    }
    for (int e = tid; e < nbk; e += kThreads) {
        const int b = owner(bound[3], B, e);
        const int32_t key0 = bound[1][b], nk = bound[1][b + 1] - key0, nq = bound[0][b + 1] - bound[0][b];
        const int32_t pos = (e - bound[3][b]) * kRows;
        // causal: token t sees key pos from t = pos - (nk - nq) on
        const int32_t t = p.causal ? max(0, pos - (nk - nq)) : 0;
        KBlock k{};
        k.key0 = key0 + pos;
        k.nkeys = min(kRows, nk - pos);
        k.pos = pos;
        k.q0 = bound[2][b] + t / tpb;
        k.nq = t < nq ? bound[2][b + 1] - k.q0 : 0;
        v.kblocks[e] = k;
    }
    __syncthreads();
    by_work(nbq, v.order_q, bins, s, [&](int e) { return v.qblocks[e].chunks; });
    if (backward) by_work(nbk, v.order_k, bins, s, [&](int e) { return v.kblocks[e].nq; });
    if (tid == 0) *v.lists = Lists{nbq, nbk, 0, 0, 0};
}

}  // namespace

cudaError_t launch_lists(const PackedProblem& p, const View& v, bool backward, int head_dim, const Tails& tails,
                         cudaStream_t stream) {
    const unsigned grid = p.clear_tail && (tails.n > 0 || tails.lse != nullptr) ? 1 + 32 : 1;
    packed_lists_kernel<<<grid, kThreads, 0, stream>>>(p, v, backward ? 1 : 0, head_dim, tails);
    return cudaGetLastError();
}

cudaError_t rows_map(CUtensorMap* m, const Rows& r, int64_t tokens, int heads, int d, int box_heads, int box_tokens) {
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
    cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(tokens)};
    cuuint64_t strides[2] = {cuuint64_t(r.hs) * 2, cuuint64_t(r.ts) * 2};
    cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_tokens)};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult c = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, r.p, dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return c == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace packed
}  // namespace sta
