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
constexpr int kBins = 1024;     // walks are ordered by min(steps, kBins - 1), falling
constexpr int kNear = 1024;     // up to this many sequences the bounds stay in shared memory

// Inclusive scans of two values over the CTA's threads with `op`: one barrier, every warp joins the
// warps' totals for itself; two buffers in turn, so that the next scan need not wait for its readers.
struct Scan {
    int2 (*sh)[32];
    int turn;
};
template <class Op>
__device__ int2 warp_scan(int2 v, const Op& op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const int32_t x = __shfl_up_sync(~0u, v.x, i), y = __shfl_up_sync(~0u, v.y, i);
        if (lane >= i) v = make_int2(op(v.x, x), op(v.y, y));
    }
    return v;
}
template <class Op>
__device__ int2 scan(int2 v, Scan& s, const Op& op) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_scan(v, op);
    if (lane == 31) s.sh[s.turn][warp] = v;
    __syncthreads();
    const int2 all = warp_scan(s.sh[s.turn][lane], op);
    s.turn ^= 1;
    const int from = warp > 0 ? warp - 1 : 0;
    const int32_t x = __shfl_sync(~0u, all.x, from), y = __shfl_sync(~0u, all.y, from);
    return warp > 0 ? make_int2(op(v.x, x), op(v.y, y)) : v;
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

constexpr int kNearBlocks = 2048;  // up to this many blocks their work and parts stay in shared memory

// Part `i` of `parts` of a walk of w steps: its first step and their number.
__device__ __forceinline__ int2 part_of(int32_t w, int32_t parts, int32_t i) {
    const int32_t each = w / parts, more = w - each * parts;
    return make_int2(i * each + min(i, more), each + (i < more ? 1 : 0));
}

// Walks of blocks 0 .. n - 1 by falling work, split into parts where `split`.  work(e): the steps
// of block e; set(e, parts, slot): writes its split and slot; put(i, e, first, n, slot): writes
// walk i.  Returns the number of walks.  Which walk runs first changes no result, so the order
// within a bin is free.
template <class Work, class Set, class Put>
__device__ int32_t make_walks(int32_t n, int32_t kv_heads, bool split, int32_t sms, int2* near, int2* scratch, int32_t* bins,
                              Scan& s, const Work& work, const Set& set, const Put& put) {
    __shared__ unsigned long long sh_total;
    __shared__ int32_t sh_most, sh_end[2];
    if (threadIdx.x == 0) {
        sh_total = 0ull;
        sh_most = 0;
    }
    bins[threadIdx.x] = 0;
    __syncthreads();
    int32_t cap = INT32_MAX;
    if (split) {
        unsigned long long mine = 0ull;
        int32_t most = 0;
        for (int e = threadIdx.x; e < n; e += kThreads) {
            mine += unsigned(work(e));
            most = max(most, work(e));
        }
        for (int i = 16; i > 0; i >>= 1) {
            mine += __shfl_xor_sync(~0u, mine, i);
            most = max(most, __shfl_xor_sync(~0u, most, i));
        }
        if (threadIdx.x % 32 == 0 && most > 0) {
            atomicAdd(&sh_total, mine);
            atomicMax(&sh_most, most);
        }
        __syncthreads();
        // nothing to split while the longest walk is below an SM's share; else into halves of a
        // share: a block of w > cap steps has fewer than 2 w / cap parts, all together fewer
        // than kSplitParts to an SM
        const unsigned long long share = sh_total * unsigned(kv_heads) / unsigned(sms);
        if (4ull * unsigned(sh_most) > 3ull * share) cap = max(kMinPart, int32_t(min(share / 2 + 1, 1ull << 30)));
        split = cap < sh_most;
    }
    const auto add_ = [](int32_t a, int32_t b) { return a + b; };
    int32_t walks = n, slots = 0;
    // whole walks are their blocks in order; else (block, part) of each are listed first
    int2* list = nullptr;
    if (split) {
        walks = 0;
        list = n + kSplitParts * sms <= kNearBlocks ? near : scratch;
        for (int e0 = 0; e0 < n; e0 += kThreads) {
            const int e = e0 + threadIdx.x;
            const int32_t w = e < n ? work(e) : 0, parts = e < n ? (w > cap ? (w + cap - 1) / cap : 1) : 0;
            const int32_t more = parts > 1 ? parts : 0;
            const int2 upto = scan(make_int2(parts, more), s, add_);
            const int32_t at = walks + upto.x - parts, slot = slots + upto.y - more;
            if (threadIdx.x == kThreads - 1) {
                sh_end[0] = at + parts;
                sh_end[1] = slot + more;
            }
            if (e < n) {
                set(e, parts, slot);
                for (int i = 0; i < parts; ++i) {
                    list[at + i] = make_int2(e, i);
                    atomicAdd(&bins[kBins - 1 - min(part_of(w, parts, i).y, kBins - 1)], 1);
                }
            }
            __syncthreads();
            walks = sh_end[0];
            slots = sh_end[1];
            __syncthreads();
        }
    } else {
        for (int e = threadIdx.x; e < n; e += kThreads) {
            set(e, 1, 0);
            atomicAdd(&bins[kBins - 1 - min(work(e), kBins - 1)], 1);
        }
    }
    __syncthreads();
    const int32_t mine = bins[threadIdx.x];
    const int32_t upto = scan(make_int2(mine, 0), s, add_).x;
    bins[threadIdx.x] = upto - mine;
    __syncthreads();
    for (int i = threadIdx.x; i < walks; i += kThreads) {
        const int2 it = split ? list[i] : make_int2(i, 0);
        const int32_t w = work(it.x), parts = w > cap ? (w + cap - 1) / cap : 1;
        const int2 p = part_of(w, parts, it.y);
        put(atomicAdd(&bins[kBins - 1 - min(p.y, kBins - 1)], 1), it.x, p.x, p.y, parts > 1, it.y);
    }
    __syncthreads();
    return walks;
}
static_assert(kBins == kThreads, "one bin for each thread in the scan");

// Zero the rows of no sequence: behind the last, and before the first (block 0 builds the lists meanwhile).
__device__ void clear_tails(const PackedProblem& p, const Tails& t, int head_dim) {
    // the last bound as block 0 cuts it: the running maximum of the clamped bounds
    __shared__ int32_t first[2], last[2];
    if (threadIdx.x < 2) first[threadIdx.x] = last[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; p.batch > 0 && i <= p.batch; i += blockDim.x) {
        const int32_t q = min(p.cu_q[i], p.tokens_q), k = min(p.cu_k[i], p.tokens_k);
        if (i == 0) {
            first[0] = max(q, 0);
            first[1] = max(k, 0);
        }
        atomicMax(&last[0], q);
        atomicMax(&last[1], k);
    }
    __syncthreads();
    const int64_t id = int64_t(blockIdx.x - 1) * blockDim.x + threadIdx.x, step = int64_t(gridDim.x - 1) * blockDim.x;
    for (int i = 0; i < t.n; ++i) {
        const int32_t before = t.is_q[i] ? first[0] : first[1], from = t.is_q[i] ? last[0] : last[1];
        const int32_t tokens = t.is_q[i] ? p.tokens_q : p.tokens_k, parts = head_dim / 8;
        const int64_t n = int64_t(before + tokens - from) * t.heads[i] * parts;
        for (int64_t j = id; j < n; j += step) {
            const int64_t row = j / parts;
            const int32_t nth = int32_t(row / t.heads[i]), h = int32_t(row % t.heads[i]);
            const int64_t tok = nth < before ? nth : from + nth - before;
            *reinterpret_cast<uint4*>(t.r[i].p + tok * t.r[i].ts + h * t.r[i].hs + (j % parts) * 8) =
                make_uint4(0u, 0u, 0u, 0u);
        }
    }
    if (t.lse != nullptr) {
        const int64_t none = first[0] + p.tokens_q - last[0];
        for (int64_t j = id; j < none * p.heads; j += step) {
            const int64_t nth = j % none;
            t.lse[(j / none) * p.tokens_q + (nth < first[0] ? nth : last[0] + nth - first[0])] = -INFINITY;
        }
    }
}

// Latency-bound: a few scans and a counting sort by one CTA, 7-12 us under a profiler, of which the
// launch of the kernels that read the lists hides a part: they start meanwhile and wait.
__global__ void __launch_bounds__(kThreads) packed_lists_kernel(const PackedProblem p, const View v, int backward,
                                                                int head_dim, const Tails tails) {
    ops::grid_launch_dependents();
    ops::grid_wait();
    if (blockIdx.x > 0) {
        clear_tails(p, tails, head_dim);
        return;
    }
    __shared__ int2 sh_scan[2][32];
    Scan s{sh_scan, 0};
    __shared__ int32_t bins[kBins];
    __shared__ int32_t near_[4][kNear + 1];
    __shared__ int32_t near_work[kNearBlocks];
    __shared__ int2 near_list[kNearBlocks];
    const int B = p.batch, tid = threadIdx.x, tpb = kRows / p.group;
    int32_t* bound[4];  // cut cu_q, cut cu_k, first query block, first key block
    for (int i = 0; i < 4; ++i) bound[i] = B <= kNear ? near_[i] : v.bounds + int64_t(i) * (B + 1);
    const auto max_ = [](int32_t a, int32_t b) { return max(a, b); };
    const auto add_ = [](int32_t a, int32_t b) { return a + b; };
    // ---- bounds cut to the tensors and made rising; blocks counted
    int32_t cq = 0, ck = 0, nbq = 0, nbk = 0;  // carried over passes of 1024 sequences
    bool cut = false;
    int32_t rq = INT32_MIN, rk = INT32_MIN;  // this thread's bounds (the first pass's are on their way with the starts)
    auto fetch = [&](int i) {
        rq = i < B ? p.cu_q[i + 1] : INT32_MIN;
        rk = i < B ? p.cu_k[i + 1] : INT32_MIN;
    };
    if (B > 0) {
        const int32_t a = p.cu_q[0], b = p.cu_k[0];
        fetch(tid);
        cq = max(0, min(a, p.tokens_q));
        ck = max(0, min(b, p.tokens_k));
        cut = a != 0 || b != 0;  // (rows before the first sequence are no one's)
    }
    if (tid == 0) {
        bound[0][0] = cq;
        bound[1][0] = ck;
        bound[2][0] = bound[3][0] = 0;
    }
    for (int i0 = 0; i0 < B; i0 += kThreads) {
        const int i = i0 + tid;
        if (i0 > 0) fetch(i);
        const int2 top = scan(make_int2(min(rq, p.tokens_q), min(rk, p.tokens_k)), s, max_);
        const int32_t hq = max(cq, top.x), hk = max(ck, top.y);
        cut |= i < B && (rq != hq || rk != hk);
        if (i < B) {
            bound[0][i + 1] = hq;
            bound[1][i + 1] = hk;
        }
        __syncthreads();
        const int32_t nq = i < B ? hq - bound[0][i] : 0, nk = i < B ? hk - bound[1][i] : 0;
        const int2 blocks = scan(make_int2((nq + tpb - 1) / tpb, (nk + kRows - 1) / kRows), s, add_);
        const int32_t bq = nbq + blocks.x, bk = backward ? nbk + blocks.y : 0;
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
        if (nbq <= kNearBlocks) near_work[e] = q.chunks;
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
    const int32_t wq = make_walks(
        nbq, p.kv_heads, v.split_q != 0, v.sms, near_list, v.scratch, bins, s,
        [&](int e) { return nbq <= kNearBlocks ? near_work[e] : v.qblocks[e].chunks; },
        [&](int e, int32_t parts, int32_t slot) {
            v.qblocks[e].split = parts;
            v.qblocks[e].slot = slot;
        },
        [&](int i, int e, int32_t first, int32_t n, bool part, int32_t which) {
            const QBlock q = v.qblocks[e];
            v.qwalks[i] = QWork{q.tok0, q.ntok, q.key0, q.nkeys, q.limit0, first, n, part ? q.slot + which : -1, e, 0, {0, 0}};
        });
    int32_t wk = 0;
    if (backward) {
        for (int e = tid; e < nbk && nbk <= kNearBlocks; e += kThreads) near_work[e] = v.kblocks[e].nq;
        __syncthreads();
        wk = make_walks(
            nbk, p.kv_heads, v.split_k != 0, v.sms, near_list, v.scratch, bins, s,
            [&](int e) { return nbk <= kNearBlocks ? near_work[e] : v.kblocks[e].nq; },
            [&](int e, int32_t parts, int32_t slot) {
                v.kblocks[e].split = parts;
                v.kblocks[e].slot = slot;
            },
            [&](int i, int e, int32_t first, int32_t n, bool part, int32_t which) {
                const KBlock k = v.kblocks[e];
                v.kwalks[i] = KWork{k.key0, k.nkeys, k.pos, k.q0 + first, n, part ? k.slot + which : -1, 0, 0};
            });
    }
    if (tid == 0) *v.lists = Lists{nbq, nbk, wq, wk, 0, 0, 0};
}

}  // namespace

cudaError_t launch_lists(const PackedProblem& p, const View& v, bool backward, int head_dim, const Tails& tails,
                         cudaStream_t stream) {
    const unsigned grid = p.clear_tail && (tails.n > 0 || tails.lse != nullptr) ? 1 + 32 : 1;
    return launch(packed_lists_kernel, dim3(grid), kThreads, 0, stream, true, p, v, backward ? 1 : 0, head_dim, tails);
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
