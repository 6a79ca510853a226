// host.cpp -- the tensor helpers of the operators around the FP8 products of a decoder layer, as a CPython
// module (_host): argument checks, outputs, workspaces and the call of the C ABI.
//
// These operators take a few microseconds on the GPU; the same checks in Python took four times as long as the
// rest of the call (a decode step of qk_norm_rope: 15.3 us a call, of it 4.3 in checks, 2.9 for the output, 1.4 for
// the argument structure and 3.7 in the ctypes call). Nothing is computed here. Every error is raised as a Python
// exception before the library is called; the library's own status becomes an Fp8bsError.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>

#include <algorithm>
#include <cmath>
#include <map>
#include <string>
#include <utility>

#include "../../include/fp8bs.h"

namespace {

struct Error {
    PyObject* type;
    std::string text;
};

[[noreturn]] void type_error(const std::string& text) { throw Error{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string& text) { throw Error{PyExc_ValueError, text}; }

struct Raised {};      // a Python exception is set already

// ------------------------------------------------------------------------------ the C ABI

PyObject* g_error_class = nullptr;      // Fp8bsError(function, status)

#define FP8BS_FUNCTIONS(X)            \
    X(qk_norm_rope)                   \
    X(paged_attention)                \
    X(paged_attention_workspace_size) \
    X(moe_route)                      \
    X(moe_experts)                    \
    X(moe_layer)                      \
    X(moe_workspace_size)
#define FP8BS_POINTER(name) decltype(&fp8bs_##name) p_##name = nullptr;
FP8BS_FUNCTIONS(FP8BS_POINTER)
#undef FP8BS_POINTER

void check_status(const char* function, int status) {
    if (status == FP8BS_OK) return;
    PyObject* e = PyObject_CallFunction(g_error_class, "si", function, status);
    if (e) {
        PyErr_SetObject(g_error_class, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

// ------------------------------------------------------------------------------ arguments

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

std::string type_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        default: return c10::toString(t);
    }
}

// Type, rank and device; dev < 0: the device is the tensor's own.
void check_tensor(const at::Tensor& t, at::ScalarType type, int64_t ndim, const char* name, int dev) {
    if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
    if (t.dim() != ndim) value_error(std::string(name) + " must be a " + std::to_string(ndim) + "-D tensor");
    if (dev >= 0 && t.get_device() != dev)
        value_error(std::string(name) + " must be on cuda:" + std::to_string(dev) + ", like the other tensors");
}

const at::Tensor& rows(PyObject* o, int64_t ndim, const char* name, int dev = -1) {
    const at::Tensor& t = tensor(o, name);
    check_tensor(t, at::kBFloat16, ndim, name, dev);
    if (t.size(ndim - 1) > 1 && t.stride(ndim - 1) != 1)
        value_error(std::string(name) + " must have contiguous rows");
    return t;
}

const at::Tensor& dense(PyObject* o, at::ScalarType type, int64_t ndim, const char* name, int dev = -1) {
    const at::Tensor& t = tensor(o, name);
    check_tensor(t, type, ndim, name, dev);
    if (!t.is_contiguous())
        value_error(std::string(name) + " must be a contiguous " + std::to_string(ndim) + "-D tensor");
    return t;
}

void check_shape(const at::Tensor& t, at::IntArrayRef shape, const char* name, const char* meaning) {
    if (t.sizes() != shape) value_error(std::string(name) + " must have the shape " + meaning);
}

bool none(PyObject* o) { return o == Py_None; }

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

// The output: new, or the caller's, a contiguous bf16 tensor of exactly this shape, on the GPU or pinned.
at::Tensor output(PyObject* out, at::IntArrayRef shape, const at::Tensor& like) {
    if (none(out)) return at::empty(shape, like.options().dtype(at::kBFloat16));
    const at::Tensor& t = tensor(out, "out");
    if (!t.is_cuda() && !t.is_pinned()) type_error("out must be a CUDA tensor or a pinned host tensor");
    if (t.scalar_type() != at::kBFloat16) type_error("out must be torch.bfloat16, got " + type_name(t.scalar_type()));
    if (!t.is_contiguous() || t.sizes() != shape) {
        std::string want;
        for (int64_t n : shape) want += (want.empty() ? "" : ", ") + std::to_string(n);
        value_error("out must be contiguous, of shape (" + want + ")");
    }
    if (t.is_cuda() && t.get_device() != like.get_device()) value_error("out must be on the device of the inputs");
    return t;
}

struct Cache {
    fp8bs_kv_cache c;
};

// A PagedCache (k, v).
Cache cache_of(PyObject* o, int dev) {
    PyObject* items = PySequence_Fast(o, "cache must be a PagedCache");
    if (!items) throw Raised{};
    struct Hold {
        PyObject* p;
        ~Hold() { Py_DECREF(p); }
    } hold{items};
    if (PySequence_Fast_GET_SIZE(items) != 2) type_error("cache must be a PagedCache");
    const at::Tensor& k = rows(PySequence_Fast_GET_ITEM(items, 0), 4, "cache.k", dev);
    const at::Tensor& v = rows(PySequence_Fast_GET_ITEM(items, 1), 4, "cache.v", dev);
    if (k.size(0) != v.size(0) || k.size(1) != v.size(1) || k.size(2) != v.size(2))
        value_error("cache.k and cache.v must have the same pages, page size and heads");
    return Cache{{k.data_ptr(), v.data_ptr(), k.size(0), k.size(1), k.size(2), k.size(3), v.size(3), k.stride(0),
                  k.stride(1), k.stride(2), v.stride(0), v.stride(1), v.stride(2)}};
}

// ------------------------------------------------------------------------------ workspaces

// Device memory for one call. Calls on a stream run one after another and share one buffer per device and stream, which
// grows by doubling (the outgrown one goes back to the allocator, which hands it out again in the stream's order). A
// call that is being captured gets memory of its own from the allocator, as an output would: the graph keeps the
// address and may be replayed on any stream, beside graphs that were captured on the same one and beside eager calls.
at::Tensor scratch(int dev, void* stream, size_t bytes, const at::Tensor& like) {
    const auto make = [&](size_t size) {
        return at::empty({static_cast<int64_t>(size)}, like.options().dtype(at::kByte));
    };
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) return make(bytes);
    static auto* all = new std::map<std::pair<int, void*>, at::Tensor>;
    at::Tensor& held = (*all)[{dev, stream}];
    const size_t have = held.defined() ? held.nbytes() : 0;
    if (have < bytes) held = make(std::max(bytes, have ? 2 * have : size_t{1} << 20));
    return held;
}

void* current_stream(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

// ------------------------------------------------------------------------------ the operators

// q, k, cos, sin, positions, q_weight, k_weight, eps, rot_start, interleaved, cache, v, slots, out
PyObject* qk_norm_rope(PyObject* const* x) {
    const at::Tensor& q = rows(x[0], 3, "q");
    const int dev = q.get_device();
    const int64_t T = q.size(0), hq = q.size(1), d = q.size(2);
    const at::Tensor& k = rows(x[1], 3, "k", dev);
    if (k.size(0) != T || k.size(2) != d) value_error("q and k must have the same tokens and channels");
    const int64_t hk = k.size(1);
    const at::Tensor& cos = dense(x[2], at::kFloat, 2, "cos", dev);
    const at::Tensor& sin = dense(x[3], at::kFloat, 2, "sin", dev);
    if (cos.sizes() != sin.sizes()) value_error("cos and sin must have the same shape");
    const at::Tensor& positions = dense(x[4], at::kInt, 1, "positions", dev);
    check_shape(positions, {T}, "positions", "[T]");
    fp8bs_qk_norm_rope_args a = {};
    for (int i = 0; i < 2; ++i) {
        if (none(x[5 + i])) continue;
        const char* name = i == 0 ? "q_weight" : "k_weight";
        const at::Tensor& w = dense(x[5 + i], at::kBFloat16, 1, name, dev);
        check_shape(w, {d}, name, "[D]");
        (i == 0 ? a.q_weight : a.k_weight) = w.data_ptr();
    }
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    at::Tensor k_out;
    if (none(x[10])) {
        if (!none(x[11]) || !none(x[12])) value_error("v and slots need a cache");
        k_out = at::empty({T, hk, d}, k.options());
        a.cache = {k_out.data_ptr(), nullptr, std::min<int64_t>(T, 1), std::max<int64_t>(T, 1), hk, d, d, 0, hk * d, d,
                   0, 0, 0};
    } else {
        if (none(x[11]) || none(x[12])) value_error("a cache needs v and slots");
        a.cache = cache_of(x[10], dev).c;
        const at::Tensor& v = rows(x[11], 3, "v", dev);
        if (a.cache.heads != hk || a.cache.dk != d) value_error("k does not match the cache's heads and channels");
        check_shape(v, {T, hk, a.cache.dv}, "v", "[T, heads, Dv] of k and the cache");
        const at::Tensor& slots = dense(x[12], at::kLong, 1, "slots", dev);
        check_shape(slots, {T}, "slots", "[T]");
        a.v = v.data_ptr();
        a.v_token_stride = v.stride(0);
        a.v_head_stride = v.stride(1);
        a.slots = slots.data_ptr<int64_t>();
    }
    at::Tensor out = output(x[13], {T, hq, d}, q);
    a.q = q.data_ptr();
    a.k = k.data_ptr();
    a.q_token_stride = q.stride(0);
    a.q_head_stride = q.stride(1);
    a.k_token_stride = k.stride(0);
    a.k_head_stride = k.stride(1);
    a.cos = cos.data_ptr<float>();
    a.sin = sin.data_ptr<float>();
    a.positions = positions.data_ptr<int32_t>();
    a.q_out = out.data_ptr();
    a.T = T;
    a.q_heads = hq;
    a.max_positions = cos.size(0);
    a.rot_start = integer(x[8]);
    a.rot_dim = 2 * cos.size(1);
    a.interleaved = truth(x[9]) ? 1 : 0;
    a.eps = static_cast<float>(real(x[7]));
    check_status("fp8bs_qk_norm_rope", p_qk_norm_rope(&a, current_stream(dev)));
    if (!k_out.defined()) return THPVariable_Wrap(std::move(out));
    PyObject* two = PyTuple_New(2);
    if (!two) throw Raised{};
    PyTuple_SET_ITEM(two, 0, THPVariable_Wrap(std::move(out)));
    PyTuple_SET_ITEM(two, 1, THPVariable_Wrap(std::move(k_out)));
    return two;
}

// q, cache, page_table, q_start, kv_len, scale, causal, window, max_q_len, max_kv_len, out, return_lse
PyObject* paged_attention(PyObject* const* x) {
    const at::Tensor& q = rows(x[0], 3, "q");
    const int dev = q.get_device();
    fp8bs_paged_attention_args a = {};
    a.cache = cache_of(x[1], dev).c;
    a.T = q.size(0);
    a.q_heads = q.size(1);
    if (q.size(2) != a.cache.dk || a.cache.heads < 1 || a.q_heads % a.cache.heads)
        value_error("q does not match the cache's channels, or its heads are no multiple");
    const at::Tensor& table = dense(x[2], at::kInt, 2, "page_table", dev);
    const at::Tensor& q_start = dense(x[3], at::kInt, 1, "q_start", dev);
    const at::Tensor& kv_len = dense(x[4], at::kInt, 1, "kv_len", dev);
    a.B = table.size(0);
    a.table_stride = table.size(1);
    if (kv_len.size(0) != a.B || q_start.size(0) != a.B + 1)
        value_error("page_table, q_start and kv_len must agree on the number of sequences");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    at::Tensor out = output(x[10], {a.T, a.q_heads, a.cache.dv}, q);
    at::Tensor lse;
    if (truth(x[11])) {
        lse = at::empty({a.T, a.q_heads}, q.options().dtype(at::kFloat));
        a.lse = lse.data_ptr<float>();
    }
    a.q = q.data_ptr();
    a.q_token_stride = q.stride(0);
    a.q_head_stride = q.stride(1);
    a.page_table = table.data_ptr<int32_t>();
    a.q_start = q_start.data_ptr<int32_t>();
    a.kv_len = kv_len.data_ptr<int32_t>();
    a.out = out.data_ptr();
    a.scale = none(x[5]) ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(a.cache.dk)))
                         : static_cast<float>(real(x[5]));
    a.causal = truth(x[6]) ? 1 : 0;
    a.window = integer(x[7]);
    a.max_q_len = none(x[8]) ? a.T : integer(x[8]);
    a.max_kv_len = none(x[9]) ? a.table_stride * a.cache.page_size : integer(x[9]);
    void* stream = current_stream(dev);
    size_t need = 0;
    check_status("fp8bs_paged_attention", p_paged_attention_workspace_size(&a, &need));
    at::Tensor work;                   // (held until the call is queued)
    if (need > 0) {
        work = scratch(dev, stream, need, q);
        a.workspace = work.data_ptr();
        a.workspace_bytes = work.nbytes();
    }
    check_status("fp8bs_paged_attention", p_paged_attention(&a, stream));
    if (!lse.defined()) return THPVariable_Wrap(std::move(out));
    PyObject* two = PyTuple_New(2);
    if (!two) throw Raised{};
    PyTuple_SET_ITEM(two, 0, THPVariable_Wrap(std::move(out)));
    PyTuple_SET_ITEM(two, 1, THPVariable_Wrap(std::move(lse)));
    return two;
}

// x[0] .. [8]: router_w, top_k, bias, score, groups, topk_groups, normalise, route_scale; for input t.
fp8bs_moe_routing routing(const at::Tensor& t, int dev, PyObject* const* x, int64_t* experts) {
    fp8bs_moe_routing r = {};
    const at::Tensor& w = dense(x[0], at::kBFloat16, 2, "router_w", dev);
    *experts = w.size(0);
    if (w.size(1) != t.size(1)) value_error("router_w must have x's channels");
    r.router_w = w.data_ptr();
    r.top_k = integer(x[1]);
    if (!none(x[2])) {
        const at::Tensor& b = dense(x[2], at::kFloat, 1, "bias", dev);
        check_shape(b, {*experts}, "bias", "[E]");
        r.bias = b.data_ptr<float>();
    }
    const char* score = PyUnicode_Check(x[3]) ? PyUnicode_AsUTF8(x[3]) : nullptr;
    if (score && std::string(score) == "sigmoid")
        r.score = FP8BS_SCORE_SIGMOID;
    else if (score && std::string(score) == "softmax")
        r.score = FP8BS_SCORE_SOFTMAX;
    else
        value_error("unknown score: \"sigmoid\" or \"softmax\"");
    r.groups = integer(x[4]);
    r.topk_groups = integer(x[5]);
    r.normalise = none(x[6]) ? r.score == FP8BS_SCORE_SIGMOID : truth(x[6]);
    r.route_scale = static_cast<float>(real(x[7]));
    return r;
}

// x, router_w, top_k, bias, score, groups, topk_groups, normalise, route_scale
PyObject* moe_route(PyObject* const* x) {
    const at::Tensor& t = dense(x[0], at::kBFloat16, 2, "x");
    const int dev = t.get_device();
    int64_t experts = 0;
    const fp8bs_moe_routing r = routing(t, dev, x + 1, &experts);
    if (r.top_k < 0) value_error("top_k must not be negative");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    at::Tensor weights = at::empty({t.size(0), r.top_k}, t.options().dtype(at::kFloat));
    at::Tensor ids = at::empty({t.size(0), r.top_k}, t.options().dtype(at::kInt));
    check_status("fp8bs_moe_route", p_moe_route(t.data_ptr(), &r, weights.data_ptr<float>(), ids.data_ptr<int32_t>(),
                                                t.size(0), t.size(1), experts, current_stream(dev)));
    PyObject* two = PyTuple_New(2);
    if (!two) throw Raised{};
    PyTuple_SET_ITEM(two, 0, THPVariable_Wrap(std::move(weights)));
    PyTuple_SET_ITEM(two, 1, THPVariable_Wrap(std::move(ids)));
    return two;
}

struct Experts {
    const void *w13, *w2;
    const float *s13, *s2;
    int64_t T, D, I, E;
};

// x[0] .. x[3]: w13, s13, w2, s2
Experts experts_of(const at::Tensor& t, int dev, PyObject* const* x) {
    const at::Tensor& w13 = dense(x[0], at::kFloat8_e4m3fn, 3, "w13", dev);
    const at::Tensor& s13 = dense(x[1], at::kFloat, 3, "s13", dev);
    const at::Tensor& w2 = dense(x[2], at::kFloat8_e4m3fn, 3, "w2", dev);
    const at::Tensor& s2 = dense(x[3], at::kFloat, 3, "s2", dev);
    Experts e = {w13.data_ptr(), w2.data_ptr(), s13.data_ptr<float>(), s2.data_ptr<float>(),
                 t.size(0), t.size(1), w2.size(2), w2.size(0)};
    check_shape(w2, {e.E, e.D, e.I}, "w2", "[E, D, I]");
    check_shape(w13, {e.E, 2 * e.I, e.D}, "w13", "[E, 2I, D]");
    check_shape(s13, {e.E, 2 * e.I / FP8BS_BLOCK, e.D / FP8BS_BLOCK}, "s13", "[E, 2I/128, D/128]");
    check_shape(s2, {e.E, e.D / FP8BS_BLOCK, e.I / FP8BS_BLOCK}, "s2", "[E, D/128, I/128]");
    return e;
}

at::Tensor expert_scratch(const Experts& e, int64_t top_k, int dev, void* stream, const at::Tensor& like) {
    size_t need = 0;
    check_status("fp8bs_moe_workspace_size", p_moe_workspace_size(e.T, e.D, e.I, e.E, top_k, &need));
    return scratch(dev, stream, need, like);
}

// x, weights, ids, w13, s13, w2, s2, scale_fmt (0 or 1), out
PyObject* moe_experts(PyObject* const* x) {
    const at::Tensor& t = dense(x[0], at::kBFloat16, 2, "x");
    const int dev = t.get_device();
    const at::Tensor& weights = dense(x[1], at::kFloat, 2, "weights", dev);
    const at::Tensor& ids = dense(x[2], at::kInt, 2, "ids", dev);
    if (ids.size(0) != t.size(0) || weights.sizes() != ids.sizes())
        value_error("weights and ids must be [T, top_k]");
    const Experts e = experts_of(t, dev, x + 3);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    at::Tensor y = output(x[8], {e.T, e.D}, t);
    void* stream = current_stream(dev);
    const at::Tensor work = expert_scratch(e, ids.size(1), dev, stream, t);
    check_status("fp8bs_moe_experts",
                 p_moe_experts(t.data_ptr(), weights.data_ptr<float>(), ids.data_ptr<int32_t>(), e.w13, e.s13, e.w2,
                               e.s2, y.data_ptr(), e.T, e.D, e.I, e.E, ids.size(1), static_cast<int>(integer(x[7])),
                               work.data_ptr(), work.nbytes(), stream));
    return THPVariable_Wrap(std::move(y));
}

// x, router_w, top_k, bias, score, groups, topk_groups, normalise, route_scale, w13, s13, w2, s2, scale_fmt, out
PyObject* moe_layer(PyObject* const* x) {
    const at::Tensor& t = dense(x[0], at::kBFloat16, 2, "x");
    const int dev = t.get_device();
    int64_t experts = 0;
    const fp8bs_moe_routing r = routing(t, dev, x + 1, &experts);
    const Experts e = experts_of(t, dev, x + 9);
    if (experts != e.E) value_error("router_w must have one row per expert");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    at::Tensor y = output(x[14], {e.T, e.D}, t);
    void* stream = current_stream(dev);
    const at::Tensor work = expert_scratch(e, r.top_k, dev, stream, t);
    check_status("fp8bs_moe_layer",
                 p_moe_layer(t.data_ptr(), &r, e.w13, e.s13, e.w2, e.s2, y.data_ptr(), e.T, e.D, e.I, e.E,
                             static_cast<int>(integer(x[13])), work.data_ptr(), work.nbytes(), stream));
    return THPVariable_Wrap(std::move(y));
}

// ------------------------------------------------------------------------------ the module

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %d", N, static_cast<int>(n));
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised&) {
        return nullptr;
    } catch (const Error& e) {
        PyErr_SetString(e.type, e.text.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// init(handle of the loaded library, Fp8bsError)
PyObject* init(PyObject*, PyObject* args) {
    PyObject *handle = nullptr, *error = nullptr;
    if (!PyArg_ParseTuple(args, "OO", &handle, &error)) return nullptr;
    void* lib = PyLong_AsVoidPtr(handle);
    if (!lib) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_OSError, "libfp8bs.so is not loaded");
        return nullptr;
    }
#define FP8BS_LOOKUP(name)                                                                  \
    p_##name = reinterpret_cast<decltype(p_##name)>(dlsym(lib, "fp8bs_" #name));            \
    if (!p_##name) {                                                                        \
        PyErr_SetString(PyExc_OSError, "fp8bs_" #name " is not in libfp8bs.so");            \
        return nullptr;                                                                     \
    }
    FP8BS_FUNCTIONS(FP8BS_LOOKUP)
#undef FP8BS_LOOKUP
    Py_XDECREF(g_error_class);
    Py_INCREF(error);
    g_error_class = error;
    Py_RETURN_NONE;
}

#define ENTRY(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {{"init", init, METH_VARARGS, nullptr},
                         ENTRY(qk_norm_rope, 14),
                         ENTRY(paged_attention, 12),
                         ENTRY(moe_route, 9),
                         ENTRY(moe_experts, 9),
                         ENTRY(moe_layer, 15),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__host() { return PyModule_Create(&module); }
