// sta_torch.cpp -- the prompt side's binding for PyTorch tensors: argument checks,
// allocation of outputs and scratch, and the call into libsta.
//
// A serving step makes these calls for every layer and the smallest kernels take a
// few microseconds, so the checks are compiled (16 prompts of 1-77 tokens, one call:
// 19 us with the checks in Python).  Every computation is libsta's; this module is
// given the addresses of its entry points, so it serves whichever build of the
// library the package has loaded.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <cmath>
#include <limits>
#include <string>

#include "sta.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

decltype(&sta_packed_workspace) f_packed_workspace;
decltype(&sta_packed_forward) f_packed_forward;
decltype(&sta_packed_backward) f_packed_backward;
decltype(&sta_cache_append) f_cache_append;
decltype(&sta_cache_workspace) f_cache_workspace;
decltype(&sta_cache_attention) f_cache_attention;
decltype(&sta_cache_extend) f_cache_extend;
py::handle g_check;  // (status, what): raises StaError unless 0

[[noreturn]] void bad(const std::string& what) { throw py::value_error(what); }

std::string shape_of(at::IntArrayRef s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

// One call into the library; the interpreter runs on while the launches are queued.
template <class F, class... A>
void call(const char* what, F f, A... args) {
    int st;
    {
        py::gil_scoped_release free;
        st = int(f(args...));
    }
    if (st != int(STA_OK)) g_check(st, what);
}

// The device and stream of one call: the tensors' device is made current, and so is the call's
// stream (`stream` is a raw handle, or -1 for the current one).  New memory is thus from the pool of
// the stream that uses it: a block that another stream has just given back may still be in use by
// what is queued there.
struct On {
    c10::cuda::CUDAGuard guard;
    c10::cuda::CUDAStream before;  // the caller's current stream
    void* handle;
    std::optional<c10::cuda::CUDAStreamGuard> side;
    On(const at::Device& d, int64_t stream)
        : guard(d), before(c10::cuda::getCurrentCUDAStream(d.index())),
          handle(stream < 0 ? static_cast<void*>(before.stream()) : reinterpret_cast<void*>(stream)) {
        if (handle != static_cast<void*>(before.stream()))
            side.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), before.device_index()));
    }
    // New tensors that the caller gets, who may use them on the current stream and drop them there.
    void keep(const Tensor& t) const {
        if (side.has_value() && t.defined() && t.numel() > 0)
            c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), before);
    }
};

at::Device cuda_device(const char* name, const Tensor& t) {
    if (!t.is_cuda()) bad(std::string(name) + " must be a CUDA tensor");
    return t.device();
}

sta_rows rows(const char* name, const Tensor& t, const at::Device& dev, int64_t tokens, int64_t heads, int64_t d) {
    if (t.scalar_type() != at::kBFloat16 || t.device() != dev) bad(std::string(name) + " must be a bf16 tensor on " + dev.str());
    if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != d)
        bad(std::string(name) + " has shape " + shape_of(t.sizes()) + ", expected " + shape_of({tokens, heads, d}));
    int64_t st = t.stride(0), sh = t.stride(1);
    if (heads == 1) sh = d;
    if (tokens <= 1) st = heads * d;
    void* p = t.data_ptr();
    if ((d > 1 && t.stride(2) != 1) || st <= 0 || sh <= 0 || (st | sh) % 8 != 0 || reinterpret_cast<uintptr_t>(p) % 16 != 0)
        bad(std::string(name) + ": the last dimension must be contiguous, the other strides positive multiples of 8 elements "
            "and the data 16-byte aligned (strides " + shape_of(t.strides()) + ")");
    return sta_rows{p, st, sh};
}

// Contiguous vector of `n` (any size if n < 0).
template <class T>
T* vec(const char* name, const Tensor& t, const at::Device& dev, int64_t n) {
    if (t.scalar_type() != c10::CppTypeToScalarType<T>::value || t.device() != dev || t.dim() != 1 || !t.is_contiguous() ||
        (n >= 0 && t.size(0) != n))
        bad(std::string(name) + " must be a contiguous " + toString(c10::CppTypeToScalarType<T>::value) + " tensor of shape [" +
            (n < 0 ? "n" : std::to_string(n)) + "] on " + dev.str());
    return static_cast<T*>(t.data_ptr());
}

float* lse_ptr(const Tensor& lse, const at::Device& dev, int64_t heads, int64_t tokens) {
    if (lse.scalar_type() != at::kFloat || lse.device() != dev || !lse.is_contiguous() || lse.dim() != 2 ||
        lse.size(0) != heads || lse.size(1) != tokens)
        bad("lse must be a contiguous fp32 tensor of shape " + shape_of({heads, tokens}) + " on " + dev.str());
    return static_cast<float*>(lse.data_ptr());
}

// New memory from the current stream's pool, within On the call's (not through the dispatcher: 0.5 us less for each).
Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const at::Device& dev) {
    return Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
}
Tensor like(const Tensor& t) { return fresh(t.sizes(), t.scalar_type(), t.device()); }

// `n` elements of a new vector from `at` on.
Tensor part(const Tensor& t, int64_t at, int64_t n) {
    auto impl = c10::make_intrusive<at::TensorImpl>(c10::Storage(t.storage()), t.key_set(), t.dtype());
    impl->set_storage_offset(at);
    impl->set_sizes_contiguous({n});
    return Tensor(std::move(impl));
}

Tensor scratch(const OptTensor& given, int64_t need, const at::Device& dev) {
    if (!given.has_value()) return need == 0 ? Tensor() : fresh({need}, at::kByte, dev);
    const Tensor& w = *given;
    if (w.device() != dev || w.scalar_type() != at::kByte || !w.is_contiguous() || w.numel() < need)
        bad("workspace must be a contiguous uint8 tensor of at least " + std::to_string(need) + " bytes on " + dev.str());
    return w;
}
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
int64_t bytes(const Tensor& t) { return t.defined() ? t.numel() : 0; }

sta_packed problem(const Tensor& q, const Tensor& k, const Tensor& cu_q, const OptTensor& cu_k, bool causal, bool clear_tail,
                   const std::optional<double>& scale, const at::Device& dev) {
    if (q.dim() != 3 || k.dim() != 3) bad("q and k must be [tokens, heads, d]");
    const int64_t batch = cu_q.dim() == 1 ? cu_q.size(0) - 1 : -1;
    if (batch < 0) bad("cu_q must be [sequences + 1]");
    for (int64_t n : {batch, q.size(1), k.size(1), q.size(2)})
        if (n > std::numeric_limits<int32_t>::max()) bad("sizes must fit 32 bits");
    const int32_t* cq = vec<int32_t>("cu_q", cu_q, dev, batch + 1);
    const int32_t* ck = cu_k.has_value() ? vec<int32_t>("cu_k", *cu_k, dev, batch + 1) : cq;
    return sta_packed{int32_t(batch), int32_t(q.size(1)), int32_t(k.size(1)), int32_t(q.size(2)), q.size(0), k.size(0),
                      cq, ck, causal ? 1 : 0, clear_tail ? 1 : 0,
                      scale.has_value() ? float(*scale) : float(1.0 / std::sqrt(double(q.size(2))))};
}

void packed_forward(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o, const Tensor& lse, const Tensor& cu_q,
                    const OptTensor& cu_k, bool causal, const std::optional<double>& scale, bool clear_tail,
                    const OptTensor& workspace, int64_t stream) {
    const at::Device dev = cuda_device("q", q);
    const sta_packed p = problem(q, k, cu_q, cu_k, causal, clear_tail, scale, dev);
    const sta_rows rq = rows("q", q, dev, p.tokens_q, p.heads, p.head_dim), ro = rows("o", o, dev, p.tokens_q, p.heads, p.head_dim),
                   rk = rows("k", k, dev, p.tokens_k, p.kv_heads, p.head_dim),
                   rv = rows("v", v, dev, p.tokens_k, p.kv_heads, p.head_dim);
    float* lp = lse_ptr(lse, dev, p.heads, p.tokens_q);
    if (p.tokens_q == 0) return;
    const On on(dev, stream);
    int64_t need = 0;
    call("sta_packed_workspace", f_packed_workspace, &p, 0, &need);
    const Tensor w = scratch(workspace, need, dev);
    call("sta_packed_forward", f_packed_forward, &p, &rq, &rk, &rv, &ro, lp, ptr(w), bytes(w), on.handle);
}

std::tuple<Tensor, Tensor> packed_attention(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu_q,
                                            const OptTensor& cu_k, bool causal, const std::optional<double>& scale,
                                            int64_t stream) {
    if (q.dim() != 3) bad("q must be [tokens, heads, d]");
    const at::Device dev = cuda_device("q", q);
    const On on(dev, stream);
    const Tensor o = like(q), lse = fresh({q.size(1), q.size(0)}, at::kFloat, dev);
    packed_forward(q, k, v, o, lse, cu_q, cu_k, causal, scale, true, std::nullopt, stream);
    on.keep(o);
    on.keep(lse);
    return {o, lse};
}

void packed_backward(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o, const Tensor& lse, const Tensor& dout,
                     const Tensor& dq, const Tensor& dk, const Tensor& dv, const Tensor& cu_q, const OptTensor& cu_k, bool causal,
                     const std::optional<double>& scale, bool clear_tail, const OptTensor& workspace, int64_t stream) {
    const at::Device dev = cuda_device("q", q);
    const sta_packed p = problem(q, k, cu_q, cu_k, causal, clear_tail, scale, dev);
    auto as_q = [&](const char* n, const Tensor& t) { return rows(n, t, dev, p.tokens_q, p.heads, p.head_dim); };
    auto as_k = [&](const char* n, const Tensor& t) { return rows(n, t, dev, p.tokens_k, p.kv_heads, p.head_dim); };
    const sta_rows rq = as_q("q", q), ro = as_q("o", o), rdo = as_q("dout", dout), rdq = as_q("dq", dq);
    const sta_rows rk = as_k("k", k), rv = as_k("v", v), rdk = as_k("dk", dk), rdv = as_k("dv", dv);
    const float* lp = lse_ptr(lse, dev, p.heads, p.tokens_q);
    if (p.tokens_q == 0 && p.tokens_k == 0) return;
    const On on(dev, stream);
    int64_t need = 0;
    call("sta_packed_workspace", f_packed_workspace, &p, 1, &need);
    const Tensor w = scratch(workspace, need, dev);
    call("sta_packed_backward", f_packed_backward, &p, &rq, &rk, &rv, &ro, &rdo, lp, &rdq, &rdk, &rdv, ptr(w), bytes(w), on.handle);
}

std::tuple<Tensor, Tensor, Tensor> packed_attention_backward(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o,
                                                             const Tensor& lse, const Tensor& dout, const Tensor& cu_q,
                                                             const OptTensor& cu_k, bool causal,
                                                             const std::optional<double>& scale, int64_t stream) {
    for (const auto& [name, t] : {std::pair{"q", q}, std::pair{"k", k}, std::pair{"v", v}}) cuda_device(name, t);
    const On on(q.device(), stream);
    const Tensor dq = like(q), dk = like(k), dv = like(v);
    packed_backward(q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, causal, scale, true, std::nullopt, stream);
    on.keep(dq);
    on.keep(dk);
    on.keep(dv);
    return {dq, dk, dv};
}

// ---------------------------------------------------------------- cache
sta_cache cache(const Tensor& kc, const Tensor& vc, const Tensor& ks, const Tensor& vs, at::Device& dev) {
    if (kc.dim() != 4 || !kc.is_cuda()) bad("k_cache must be a CUDA tensor [blocks, kv_heads, block_tokens, d]");
    dev = kc.device();
    auto codes = [&](const char* n, const Tensor& t) {
        if ((t.scalar_type() != at::kFloat8_e4m3fn && t.scalar_type() != at::kByte) || t.device() != dev ||
            t.sizes() != kc.sizes() || !t.is_contiguous())
            bad(std::string(n) + " must be a contiguous e4m3 (or uint8) tensor of shape " + shape_of(kc.sizes()) + " on " + dev.str());
        return t.data_ptr();
    };
    auto scales = [&](const char* n, const Tensor& t) {
        if (t.scalar_type() != at::kFloat || t.device() != dev || t.dim() != 2 || t.size(0) != kc.size(0) ||
            t.size(1) != kc.size(1) || !t.is_contiguous())
            bad(std::string(n) + " must be a contiguous fp32 tensor of shape " + shape_of({kc.size(0), kc.size(1)}) + " on " + dev.str());
        return static_cast<float*>(t.data_ptr());
    };
    for (int64_t n : kc.sizes())
        if (n > std::numeric_limits<int32_t>::max()) bad("sizes must fit 32 bits");
    return sta_cache{int32_t(kc.size(0)), int32_t(kc.size(2)), int32_t(kc.size(1)), int32_t(kc.size(3)),
                     codes("k_cache", kc), codes("v_cache", vc), scales("k_scales", ks), scales("v_scales", vs)};
}

struct Tables {
    int32_t* p;
    int32_t width;
    int64_t stride;
};
Tables tables(const Tensor& t, int64_t batch, const at::Device& dev) {
    const int64_t width = t.dim() == 2 ? t.size(1) : 0;
    if (t.scalar_type() != at::kInt || t.device() != dev || width == 0 || width > std::numeric_limits<int32_t>::max() ||
        t.size(0) != batch || (width > 1 && t.stride(1) != 1) || (batch > 1 && t.stride(0) < width))
        bad("block_tables must be an int32 tensor [" + std::to_string(batch) + ", width] on " + dev.str() + " with contiguous rows");
    return Tables{static_cast<int32_t*>(t.data_ptr()), int32_t(width), batch > 1 ? t.stride(0) : width};
}

void cache_append(const Tensor& k, const Tensor& v, const Tensor& slots, const Tensor& kc, const Tensor& vc, const Tensor& ks,
                  const Tensor& vs, int64_t stream) {
    at::Device dev(at::kCPU);
    const sta_cache c = cache(kc, vc, ks, vs, dev);
    const int64_t* sp = vec<int64_t>("slots", slots, dev, -1);
    const int64_t n = slots.size(0);
    const sta_rows rk = rows("k", k, dev, n, c.kv_heads, c.head_dim), rv = rows("v", v, dev, n, c.kv_heads, c.head_dim);
    const On on(dev, stream);
    call("sta_cache_append", f_cache_append, &c, &rk, &rv, n, sp, on.handle);
}

std::tuple<Tensor, Tensor> cache_attention(const Tensor& q, const Tensor& kc, const Tensor& vc, const Tensor& ks,
                                           const Tensor& vs, const Tensor& block_tables, const Tensor& lengths,
                                           const OptTensor& cu_q, const std::optional<double>& scale, const OptTensor& o_given,
                                           const OptTensor& lse_given, const OptTensor& workspace, int64_t stream) {
    at::Device dev(at::kCPU);
    const sta_cache c = cache(kc, vc, ks, vs, dev);
    if (q.dim() != 3) bad("q must be [tokens, heads, d]");
    const int64_t T = q.size(0), H = q.size(1), d = q.size(2);
    const int32_t* lp = vec<int32_t>("lengths", lengths, dev, -1);
    const int64_t B = lengths.size(0);
    if (B > std::numeric_limits<int32_t>::max() || H > std::numeric_limits<int32_t>::max()) bad("sizes must fit 32 bits");
    const int32_t* cp = cu_q.has_value() ? vec<int32_t>("cu_q", *cu_q, dev, B + 1) : nullptr;
    if (cp == nullptr && T != B) bad(std::to_string(T) + " queries for " + std::to_string(B) + " sequences: give cu_q");
    const Tables t = tables(block_tables, B, dev);
    const On on(dev, stream);
    const bool new_o = !o_given.has_value(), new_lse = !lse_given.has_value();
    const Tensor o = new_o ? fresh(q.sizes(), at::kBFloat16, dev) : *o_given;
    const Tensor lse = new_lse ? fresh({H, T}, at::kFloat, dev) : *lse_given;
    // (the call clears the rows of no sequence in both or in neither)
    const sta_packed p{int32_t(B), int32_t(H), c.kv_heads, int32_t(d), T, 0, cp, nullptr, 1, new_o && new_lse ? 1 : 0,
                       scale.has_value() ? float(*scale) : float(1.0 / std::sqrt(double(d)))};
    const sta_rows rq = rows("q", q, dev, T, H, d), ro = rows("o", o, dev, T, H, d);
    float* lsp = lse_ptr(lse, dev, H, T);
    if (new_o) on.keep(o);
    if (new_lse) on.keep(lse);
    if (T == 0) return {o, lse};
    if (new_o && !new_lse) o.zero_();
    if (new_lse && !new_o) lse.fill_(-INFINITY);
    int64_t need = 0;
    call("sta_cache_workspace", f_cache_workspace, &c, &p, &need);
    const Tensor w = scratch(workspace, need, dev);
    call("sta_cache_attention", f_cache_attention, &c, &p, lp, t.p, t.width, t.stride, &rq, &ro, lsp, ptr(w), bytes(w), on.handle);
    return {o, lse};
}

// (slots, cu_new, lengths, free_count, short)
std::tuple<Tensor, Tensor, Tensor, Tensor, Tensor> cache_extend(const Tensor& new_tokens, const Tensor& lengths,
                                                                const Tensor& block_tables, const Tensor& free_blocks,
                                                                const Tensor& free_count, int64_t block_tokens,
                                                                int64_t max_slots, bool in_place, int64_t stream) {
    const at::Device dev = cuda_device("lengths", lengths);
    int32_t* lp = vec<int32_t>("lengths", lengths, dev, -1);
    const int64_t B = lengths.size(0);
    if (B > std::numeric_limits<int32_t>::max() || free_blocks.numel() > std::numeric_limits<int32_t>::max() ||
        std::abs(block_tokens) > std::numeric_limits<int32_t>::max())
        bad("sizes must fit 32 bits");
    const int32_t* np = vec<int32_t>("new_tokens", new_tokens, dev, B);
    int32_t* fp = vec<int32_t>("free_blocks", free_blocks, dev, -1);
    int32_t* cp = vec<int32_t>("free_count", free_count, dev, 1);
    const Tables t = tables(block_tables, B, dev);
    const On on(dev, stream);
    // the small ones lie in one allocation
    const Tensor slots = fresh({std::max<int64_t>(max_slots, 0)}, at::kLong, dev), small = fresh({2 * B + 3}, at::kInt, dev);
    const Tensor cu = part(small, 0, B + 1), brief = part(small, B + 1, 1);
    const Tensor len_out = in_place ? lengths : part(small, B + 3, B), count_out = in_place ? free_count : part(small, B + 2, 1);
    call("sta_cache_extend", f_cache_extend, int32_t(B), int32_t(block_tokens), np, lp, static_cast<int32_t*>(len_out.data_ptr()), t.p, t.width,
                         t.stride, fp, int32_t(free_blocks.size(0)), cp, static_cast<int32_t*>(count_out.data_ptr()),
                         static_cast<int64_t*>(slots.data_ptr()), max_slots, static_cast<int32_t*>(cu.data_ptr()),
                         static_cast<int32_t*>(brief.data_ptr()), on.handle);
    on.keep(slots);
    on.keep(small);
    return {slots, cu, len_out, count_out, brief};
}

// Addresses of the loaded library's entry points, by name, and the status check.
void bind(const py::dict& at, const py::object& check_) {
    auto get = [&](const char* name) { return reinterpret_cast<void*>(py::cast<uintptr_t>(at[name])); };
    f_packed_workspace = reinterpret_cast<decltype(f_packed_workspace)>(get("sta_packed_workspace"));
    f_packed_forward = reinterpret_cast<decltype(f_packed_forward)>(get("sta_packed_forward"));
    f_packed_backward = reinterpret_cast<decltype(f_packed_backward)>(get("sta_packed_backward"));
    f_cache_append = reinterpret_cast<decltype(f_cache_append)>(get("sta_cache_append"));
    f_cache_workspace = reinterpret_cast<decltype(f_cache_workspace)>(get("sta_cache_workspace"));
    f_cache_attention = reinterpret_cast<decltype(f_cache_attention)>(get("sta_cache_attention"));
    f_cache_extend = reinterpret_cast<decltype(f_cache_extend)>(get("sta_cache_extend"));
    g_check = check_.inc_ref();  // for the life of the process
}

}  // namespace

PYBIND11_MODULE(_sta_torch, m) {
    m.attr("built_for") = STA_TORCH_KEY;
    m.def("bind", &bind);
    m.def("packed_forward", &packed_forward);
    m.def("packed_attention", &packed_attention);
    m.def("packed_backward", &packed_backward);
    m.def("packed_attention_backward", &packed_attention_backward);
    m.def("cache_append", &cache_append);
    m.def("cache_attention", &cache_attention);
    m.def("cache_extend", &cache_extend);
}
