// moe_torch.cpp -- the holders' calls on torch tensors, as a CPython extension.
//
// A small operator's call from Python costs more on the host than on the GPU: 2-3 us
// on the GPU against 14 us for the checks, the output tensors, the converted arguments
// and the launch, each a Python call of its own.  Here they are one, which takes
// 4-5 us.  Argument checks, output tensors and streams only: the library's C
// functions are called by the addresses that bind() was given.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe.h"

namespace {

decltype(&moe_topk) g_topk;
decltype(&moe_matvec) g_matvec;
decltype(&moe_experts) g_experts;
decltype(&moe_forward) g_forward;
decltype(&moe_norm) g_norm;
decltype(&moe_lora_workspace_bytes) g_lora_workspace_bytes;
decltype(&moe_lora_checked) g_lora;
PyObject* g_check;   // raises a status's error

struct Raised {};    // a Python exception is set
[[noreturn]] void raise(PyObject* type, const char* what) {
    PyErr_SetString(type, what);
    throw Raised{};
}

// A tensor argument, or null for None.
const at::Tensor* tensor(PyObject* o) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "a tensor is expected");
    return &THPVariable_Unpack(o);
}
const at::Tensor& some_tensor(PyObject* o) {
    const at::Tensor* t = tensor(o);
    if (!t) raise(PyExc_TypeError, "a tensor is expected");
    return *t;
}
long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
template <typename T> T* address(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised{};
    return static_cast<T*>(p);
}
template <typename T> T* data(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

// The current GPU: t is on it, or in pinned host memory.
int current_gpu(const at::Tensor& t) {
    if (!t.is_cuda() && !t.is_pinned()) raise(PyExc_ValueError, "tensors are on the GPU or in pinned host memory");
    const int dev = c10::cuda::current_device();
    if (t.is_cuda() && t.get_device() != dev) raise(PyExc_ValueError, "a tensor is on another device than the current one");
    return dev;
}
moe_stream_t stream_of(PyObject* o, int dev) {
    return o == Py_None ? (moe_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream()
                        : address<std::remove_pointer_t<moe_stream_t>>(o);
}
// An output on the current GPU, dev, for a call on stream st: its memory is that stream's, so that it is
// not handed out again while the call runs, and in use on the current one, where the caller reads it.
// (Made without torch's dispatcher, which at::empty goes through: 0.9 us less of some 1.8 for each output.)
at::Tensor matrix(int64_t rows, int64_t cols, at::ScalarType type, int dev, moe_stream_t st) {
    auto empty = [&] {
        const int64_t sizes[] = {rows, cols};
        return at::Tensor(at::detail::empty_generic(sizes, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                    type, std::nullopt));
    };
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev);
    if (current.stream() == st) return empty();
    const c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(st, (c10::DeviceIndex)dev));
    at::Tensor t = empty();
    c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current);
    return t;
}
int type_code(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return MOE_F32;
        case at::kBFloat16: return MOE_BF16;
        case at::kHalf: return MOE_F16;
        default: return -1;
    }
}
void check(moe_status_t s) {
    if (s == MOE_OK) return;
    PyObject* r = PyObject_CallFunction(g_check, "i", (int)s);
    if (r) {
        Py_DECREF(r);
        PyErr_SetString(PyExc_RuntimeError, "a call failed");
    }
    throw Raised{};
}
PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

void need(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) raise(PyExc_TypeError, "wrong number of arguments");
}

// bind(moe_topk, moe_matvec, moe_experts, moe_forward, moe_norm, moe_lora_workspace_bytes, moe_lora_checked, check): the
// functions' addresses.
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
    need(n, 8);
    g_topk = reinterpret_cast<decltype(g_topk)>(address<void>(a[0]));
    g_matvec = reinterpret_cast<decltype(g_matvec)>(address<void>(a[1]));
    g_experts = reinterpret_cast<decltype(g_experts)>(address<void>(a[2]));
    g_forward = reinterpret_cast<decltype(g_forward)>(address<void>(a[3]));
    g_norm = reinterpret_cast<decltype(g_norm)>(address<void>(a[4]));
    g_lora_workspace_bytes = reinterpret_cast<decltype(g_lora_workspace_bytes)>(address<void>(a[5]));
    g_lora = reinterpret_cast<decltype(g_lora)>(address<void>(a[6]));
    Py_INCREF(a[7]);
    Py_XDECREF(g_check);
    g_check = a[7];
    Py_RETURN_NONE;
}

void check_routes(const at::Tensor& t, at::ScalarType type, int64_t n, int64_t k, int dev) {
    if (t.scalar_type() != type || t.dim() != 2 || t.size(0) < n || t.size(1) != k || !t.is_contiguous() ||
        !t.is_cuda() || t.get_device() != dev)
        raise(PyExc_ValueError, "idx is int32 and w float32, contiguous [>= n, k] on the current device");
}

// topk(config address, bias or None, logits, idx or None, w or None, stream or None) -> (idx, w)
PyObject* topk(PyObject* const* a, Py_ssize_t na) {
    need(na, 6);
    moe_topk_config_t c = *address<const moe_topk_config_t>(a[0]);
    const at::Tensor* bias = tensor(a[1]);
    const at::Tensor& l = some_tensor(a[2]);
    const at::Tensor *gi = tensor(a[3]), *gw = tensor(a[4]);
    const int64_t E = c.num_experts, k = c.top_k;
    c.logits_type = type_code(l);
    if (c.logits_type < 0) raise(PyExc_KeyError, "logits are float32, bfloat16 or float16");
    if (l.dim() != 2 || l.size(1) != E || (E > 1 && l.stride(1) != 1))
        raise(PyExc_ValueError, "logits are [n, num_experts] with contiguous rows");
    if (bias && (bias->scalar_type() != at::kFloat || bias->dim() != 1 || bias->size(0) != E || !bias->is_contiguous()))
        raise(PyExc_ValueError, "bias is contiguous float32 [num_experts]");
    const int dev = current_gpu(l);
    if (bias && (!bias->is_cuda() || bias->get_device() != dev)) raise(PyExc_ValueError, "bias is not on the current device");
    const int64_t n = l.size(0);
    if (gi) check_routes(*gi, at::kInt, n, k, dev);
    if (gw) check_routes(*gw, at::kFloat, n, k, dev);
    const moe_stream_t st = stream_of(a[5], dev);
    at::Tensor idx = gi ? *gi : matrix(n, k, at::kInt, dev, st), w = gw ? *gw : matrix(n, k, at::kFloat, dev, st);
    if (n > INT32_MAX) raise(PyExc_ValueError, "too many rows");
    const void* lp = l.data_ptr();
    const float* bp = bias ? data<const float>(*bias) : nullptr;
    int32_t* ip = data<int32_t>(idx);
    float* wp = data<float>(w);
    const int64_t stride = n > 1 ? l.stride(0) : E;
    moe_status_t s;
    Py_BEGIN_ALLOW_THREADS;
    s = g_topk(&c, lp, stride, bp, (int32_t)n, ip, wp, st);
    Py_END_ALLOW_THREADS;
    check(s);
    return Py_BuildValue("(NN)", wrap(std::move(idx)), wrap(std::move(w)));
}

// matvec(config address, matrix address, bias address, the weights' device, x, out or None, stream or None) -> out
PyObject* matvec(PyObject* const* a, Py_ssize_t na) {
    need(na, 7);
    moe_matvec_config_t c = *address<const moe_matvec_config_t>(a[0]);
    const moe_qmat_t* q = address<const moe_qmat_t>(a[1]);
    const float* bias = address<const float>(a[2]);
    const long long wdev = integer(a[3]);
    const at::Tensor& x = some_tensor(a[4]);
    const at::Tensor* given = tensor(a[5]);
    const int64_t K = c.in_features, O = c.out_features;
    c.x_type = type_code(x);
    if (c.x_type != MOE_BF16 && c.x_type != MOE_F16) raise(PyExc_KeyError, "x is bfloat16 or float16");
    if (x.dim() != 2 || x.size(1) != K || x.stride(1) != 1) raise(PyExc_ValueError, "x is [n, in] with contiguous rows");
    const int dev = current_gpu(x);
    if (wdev != dev) raise(PyExc_ValueError, "the weights are not on the current device");
    const int64_t n = x.size(0);
    if (n > INT32_MAX) raise(PyExc_ValueError, "too many rows");
    const moe_stream_t st = stream_of(a[6], dev);
    int64_t ostride = O;
    at::Tensor out;
    if (given) {
        current_gpu(*given);
        if (given->dim() != 2 || given->size(0) != n || given->size(1) != O || type_code(*given) != c.out_type ||
            (O > 1 && given->stride(1) != 1))
            raise(PyExc_ValueError, "out is [n, out] of out_dtype with contiguous rows");
        out = *given;
        if (n > 1) ostride = out.stride(0);
    } else {
        if (c.accumulate) raise(PyExc_ValueError, "accumulate needs out");
        const at::ScalarType type = c.out_type == MOE_F32 ? at::kFloat : c.out_type == MOE_BF16 ? at::kBFloat16 : at::kHalf;
        out = matrix(n, O, type, dev, st);
    }
    const void* xp = x.data_ptr();
    void* op = out.data_ptr();
    const int64_t stride = n > 1 ? x.stride(0) : K;
    moe_status_t s;
    Py_BEGIN_ALLOW_THREADS;
    s = g_matvec(&c, q, bias, xp, stride, (int32_t)n, op, ostride, st);
    Py_END_ALLOW_THREADS;
    check(s);
    return wrap(std::move(out));
}

// What moe_experts and moe_forward read and write, as the library takes it.
// Outputs and routes may be device addresses, which the caller answers for.
bool is_address(PyObject* o) { return PyLong_Check(o) && !PyBool_Check(o); }
int64_t layer_rows(const moe_config_t& c, const at::Tensor& x) {
    if (x.dim() < 1 || x.size(0) > INT32_MAX) raise(PyExc_ValueError, "x is [n, hidden]");
    const int64_t n = x.size(0);
    if (x.scalar_type() != at::kBFloat16 || x.numel() != n * c.hidden || !x.is_contiguous())
        raise(PyExc_ValueError, "x is contiguous bfloat16 [n, hidden]");
    return n;
}
template <typename T>
T* layer_routes(PyObject* o, at::ScalarType type, int64_t n, int64_t k, int dev) {
    if (is_address(o)) return address<T>(o);
    const at::Tensor& t = some_tensor(o);
    if (t.scalar_type() != type || t.numel() < n * k || (t.dim() != 1 && (t.dim() != 2 || t.size(1) != k)) ||
        !t.is_contiguous() || !t.is_cuda() || t.get_device() != dev)
        raise(PyExc_ValueError, "idx is int32 and w float32, contiguous [>= n, k] on the current device");
    return data<T>(t);
}
void* layer_out(const moe_config_t& c, PyObject* o, int64_t n) {
    if (is_address(o)) return address<void>(o);
    const at::Tensor& t = some_tensor(o);
    current_gpu(t);
    if (t.scalar_type() != at::kBFloat16 || t.numel() < n * c.hidden || !t.is_contiguous())
        raise(PyExc_ValueError, "out is contiguous bfloat16 [>= n, hidden]");
    return t.data_ptr();
}

void* workspace(PyObject* o, size_t bytes, int dev) {
    if (is_address(o)) return address<void>(o);
    const at::Tensor& t = some_tensor(o);
    if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous() || t.nbytes() < bytes)
        raise(PyExc_ValueError, "the workspace is ws_bytes of contiguous memory on the current device");
    return t.data_ptr();
}

// experts(config address, weights address, workspace or its address, its bytes, x, idx, w, stream or None) -> out
PyObject* experts(PyObject* const* a, Py_ssize_t na) {
    need(na, 8);
    const moe_config_t* c = address<const moe_config_t>(a[0]);
    const moe_weights_t* wts = address<const moe_weights_t>(a[1]);
    const size_t ws_bytes = (size_t)integer(a[3]);
    const at::Tensor& x = some_tensor(a[4]);
    if (c->accumulate) raise(PyExc_ValueError, "experts() makes its output: accumulate into the out of forward()");
    const int64_t n = layer_rows(*c, x);
    const int dev = current_gpu(x);
    void* ws = workspace(a[2], ws_bytes, dev);
    const int32_t* ip = layer_routes<int32_t>(a[5], at::kInt, n, c->top_k, dev);
    const float* wp = layer_routes<float>(a[6], at::kFloat, n, c->top_k, dev);
    const moe_stream_t st = stream_of(a[7], dev);
    at::Tensor out = matrix(n, c->hidden, at::kBFloat16, dev, st);
    const void* xp = x.data_ptr();
    void* op = out.data_ptr();
    moe_status_t s;
    Py_BEGIN_ALLOW_THREADS;
    s = g_experts(c, wts, xp, (int32_t)n, ip, wp, op, ws, ws_bytes, st);
    Py_END_ALLOW_THREADS;
    check(s);
    return wrap(std::move(out));
}

// forward(config address, weights address, workspace or its address, its bytes, x, out or None, idx or None, w or None,
// whether idx and w are wanted, stream or None) -> (out, idx, w)
PyObject* forward(PyObject* const* a, Py_ssize_t na) {
    need(na, 10);
    const moe_config_t* c = address<const moe_config_t>(a[0]);
    const moe_weights_t* wts = address<const moe_weights_t>(a[1]);
    const size_t ws_bytes = (size_t)integer(a[3]);
    const at::Tensor& x = some_tensor(a[4]);
    const int routing = PyObject_IsTrue(a[8]);
    if (routing < 0) throw Raised{};
    if (a[5] == Py_None && c->accumulate) raise(PyExc_ValueError, "accumulate needs out");
    const int64_t n = layer_rows(*c, x);
    const int dev = current_gpu(x);
    void* ws = workspace(a[2], ws_bytes, dev);
    const moe_stream_t st = stream_of(a[9], dev);
    // What is not given is made here, and returned; what is given is returned as it is.
    at::Tensor out, idx, w;
    void* op;
    int32_t* ip = nullptr;
    float* wp = nullptr;
    if (a[5] != Py_None) op = layer_out(*c, a[5], n);
    if (a[6] != Py_None) ip = layer_routes<int32_t>(a[6], at::kInt, n, c->top_k, dev);
    if (a[7] != Py_None) wp = layer_routes<float>(a[7], at::kFloat, n, c->top_k, dev);
    if (a[5] == Py_None) op = (out = matrix(n, c->hidden, at::kBFloat16, dev, st)).data_ptr();
    if (a[6] == Py_None && routing) ip = data<int32_t>(idx = matrix(n, c->top_k, at::kInt, dev, st));
    if (a[7] == Py_None && routing) wp = data<float>(w = matrix(n, c->top_k, at::kFloat, dev, st));
    const void* xp = x.data_ptr();
    moe_status_t s;
    Py_BEGIN_ALLOW_THREADS;
    s = g_forward(c, wts, xp, (int32_t)n, op, ip, wp, ws, ws_bytes, st);
    Py_END_ALLOW_THREADS;
    check(s);
    auto give = [](at::Tensor& made, PyObject* given) { return made.defined() ? wrap(std::move(made)) : Py_NewRef(given); };
    return Py_BuildValue("(NNN)", give(out, a[5]), give(idx, a[6]), give(w, a[7]));
}

// A matrix [n, cols] of contiguous rows and its stride; `what` is said of any other.
struct Rows {
    void* p = nullptr;
    int64_t stride = 0;
};
Rows rows_of(const at::Tensor& t, int64_t n, int64_t cols, at::ScalarType type, const char* what) {
    if (t.dim() != 2 || t.size(0) != n || t.size(1) != cols || t.scalar_type() != type || (cols > 1 && t.stride(1) != 1))
        raise(PyExc_ValueError, what);
    return {t.data_ptr(), n > 1 ? t.stride(0) : cols};
}
at::ScalarType torch_type(int code) { return code == MOE_F32 ? at::kFloat : code == MOE_BF16 ? at::kBFloat16 : at::kHalf; }

// norm(config address, weight, whether an 8-bit output is wanted, x, residual, residual_out, out, out8, scale, stream; the last
// six may be None) -> (out, residual_out, out8, scale)
PyObject* norm(PyObject* const* a, Py_ssize_t na) {
    need(na, 10);
    moe_norm_config_t c = *address<const moe_norm_config_t>(a[0]);
    const at::Tensor& w = some_tensor(a[1]);
    const int want8 = PyObject_IsTrue(a[2]);
    if (want8 < 0) throw Raised{};
    const at::Tensor &x = some_tensor(a[3]), *res = tensor(a[4]), *gro = tensor(a[5]), *gy = tensor(a[6]), *gq = tensor(a[7]),
                     *gs = tensor(a[8]);
    const int64_t H = c.hidden;
    const bool want = c.out_type >= 0;
    c.x_type = type_code(x);
    if (c.x_type < 0) raise(PyExc_KeyError, "x is float32, bfloat16 or float16");
    if (x.dim() != 2 || x.size(1) != H || (H > 1 && x.stride(1) != 1)) raise(PyExc_ValueError, "x is [n, hidden] with contiguous rows");
    const int64_t n = x.size(0);
    if (n > INT32_MAX) raise(PyExc_ValueError, "too many rows");
    if ((gy && !want) || ((gq || gs) && !want8) || (gro && !res)) raise(PyExc_ValueError, "an output is given that is not asked for");
    c.residual_type = res ? type_code(*res) : c.x_type;
    if (res && c.residual_type != c.x_type && c.residual_type != MOE_F32)
        raise(PyExc_ValueError, "residual is of x's type or float32");
    const int64_t groups = c.scale_group ? (H + c.scale_group - 1) / c.scale_group : 1;
    Rows R, RO, Y, Q;
    const Rows X{x.data_ptr(), n > 1 ? x.stride(0) : H};
    if (res) R = rows_of(*res, n, H, torch_type(c.residual_type), "residual is [n, hidden] with contiguous rows");
    if (gro) RO = rows_of(*gro, n, H, torch_type(c.residual_type), "residual_out is [n, hidden] of the residual's type with contiguous rows");
    if (gy) Y = rows_of(*gy, n, H, torch_type(c.out_type), "out is [n, hidden] of out_dtype with contiguous rows");
    if (gq) Q = rows_of(*gq, n, H, at::kFloat8_e4m3fn, "out8 is float8_e4m3fn [n, hidden] with contiguous rows");
    if (gs && (gs->dim() != 2 || gs->size(0) != n || gs->size(1) != groups || gs->scalar_type() != at::kFloat || !gs->is_contiguous()))
        raise(PyExc_ValueError, "scale is contiguous float32 [n, groups]");
    const int dev = current_gpu(x);
    if (type_code(w) != c.weight_type || w.numel() != H || !w.is_contiguous())
        raise(PyExc_ValueError, "the weight is no longer what the operator was made with");
    if (!w.is_cuda() || w.get_device() != dev) raise(PyExc_ValueError, "the weight is not on the current device");
    for (const at::Tensor* t : {res, gro, gy, gq, gs})
        if (t) current_gpu(*t);
    const moe_stream_t st = stream_of(a[9], dev);
    at::Tensor ro, y, q, s;
    auto make = [&](int64_t cols, at::ScalarType type, at::Tensor& t) {
        t = matrix(n, cols, type, dev, st);
        return Rows{t.data_ptr(), cols};
    };
    if (res && !gro) RO = make(H, torch_type(c.residual_type), ro);
    if (want && !gy) Y = make(H, torch_type(c.out_type), y);
    if (want8 && !gq) Q = make(H, at::kFloat8_e4m3fn, q);
    float* sp = gs ? data<float>(*gs) : nullptr;
    if (want8 && !gs) sp = static_cast<float*>(make(groups, at::kFloat, s).p);
    const void* wp = w.data_ptr();
    moe_status_t status;
    Py_BEGIN_ALLOW_THREADS;
    status = g_norm(&c, X.p, X.stride, R.p, R.stride, wp, (int32_t)n, RO.p, RO.stride, Y.p, Y.stride, Q.p, Q.stride, sp, st);
    Py_END_ALLOW_THREADS;
    check(status);
    auto give = [](at::Tensor& made, PyObject* given) { return made.defined() ? wrap(std::move(made)) : Py_NewRef(given); };
    return Py_BuildValue("(NNNN)", give(y, a[6]), give(ro, a[5]), give(q, a[7]), give(s, a[8]));
}

// lora(config address, (a, b, scale or None, errors), the adapters' device, x, idx, base or None, out or None, stream or None) -> out
PyObject* lora(PyObject* const* a, Py_ssize_t na) {
    need(na, 8);
    const moe_lora_config_t* c = address<const moe_lora_config_t>(a[0]);
    if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 4) raise(PyExc_TypeError, "four tensors are expected");
    const at::Tensor &wa = some_tensor(PyTuple_GET_ITEM(a[1], 0)), &wb = some_tensor(PyTuple_GET_ITEM(a[1], 1)),
                     *scale = tensor(PyTuple_GET_ITEM(a[1], 2)), &errors = some_tensor(PyTuple_GET_ITEM(a[1], 3));
    const long long wdev = integer(a[2]);
    const at::Tensor &x = some_tensor(a[3]), &idx = some_tensor(a[4]), *base = tensor(a[5]), *given = tensor(a[6]);
    const int64_t K = c->in_features, O = c->out_features;
    if (x.dim() != 2 || x.size(1) != K || x.stride(1) != 1 || type_code(x) != c->x_type)
        raise(PyExc_ValueError, "x is [n, in] of the adapters' type with contiguous rows");
    const int64_t n = x.size(0);
    if (n > INT32_MAX) raise(PyExc_ValueError, "too many rows");
    const at::ScalarType type = torch_type(c->out_type);
    Rows Y0, Y;
    if (base) Y0 = rows_of(*base, n, O, type, "base is [n, out] of out_dtype with contiguous rows");
    if (given) Y = rows_of(*given, n, O, type, "out is [n, out] of out_dtype with contiguous rows");
    const int dev = current_gpu(x);
    const int64_t L = c->num_adapters, r = c->rank;
    if (type_code(wa) != c->x_type || type_code(wb) != c->x_type || wa.numel() != L * r * K || wb.numel() != L * r * O ||
        !wa.is_contiguous() || !wb.is_contiguous() ||
        (scale && (scale->scalar_type() != at::kFloat || scale->numel() != L || !scale->is_contiguous())))
        raise(PyExc_ValueError, "the adapters are no longer what the operator was made with");
    if (wdev != dev || wa.get_device() != dev || wb.get_device() != dev || (scale && scale->get_device() != dev) || errors.get_device() != dev)
        raise(PyExc_ValueError, "the adapters are not on the current device");
    if (idx.scalar_type() != at::kInt || idx.dim() != 1 || idx.size(0) != n || !idx.is_contiguous() || !idx.is_cuda() ||
        idx.get_device() != dev)
        raise(PyExc_ValueError, "idx is contiguous int32 [n] on the current device");
    for (const at::Tensor* t : {base, given})
        if (t) current_gpu(*t);
    const moe_stream_t st = stream_of(a[7], dev);
    at::Tensor out;
    if (given) {
        out = *given;
    } else {
        out = matrix(n, O, type, dev, st);
        Y = {out.data_ptr(), O};
    }
    // The call's own workspace, of its stream's memory: calls on several streams share none.  (One of 256
    // bytes is not used: any address will do.)
    const size_t ws_bytes = g_lora_workspace_bytes(c, (int32_t)n);
    at::Tensor ws;
    void* wp = const_cast<void*>(wa.data_ptr());
    if (ws_bytes > 256) wp = (ws = matrix(1, (int64_t)ws_bytes, at::kByte, dev, st)).data_ptr();
    const void *ap = wa.data_ptr(), *bp = wb.data_ptr(), *xp = x.data_ptr();
    const float* sp = scale ? data<const float>(*scale) : nullptr;
    const int32_t* ip = data<const int32_t>(idx);
    void* ep = errors.data_ptr();
    const int64_t stride = n > 1 ? x.stride(0) : K;
    moe_status_t s;
    Py_BEGIN_ALLOW_THREADS;
    s = g_lora(c, ap, bp, sp, xp, stride, ip, (int32_t)n, Y0.p, Y0.stride, Y.p, Y.stride, wp, ws_bytes, ep, st);
    Py_END_ALLOW_THREADS;
    check(s);
    return wrap(std::move(out));
}

// No C++ exception leaves a Python call.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(args, n);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<bind>)), METH_FASTCALL, nullptr},
    {"topk", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<topk>)), METH_FASTCALL, nullptr},
    {"matvec", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<matvec>)), METH_FASTCALL, nullptr},
    {"experts", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<experts>)), METH_FASTCALL, nullptr},
    {"forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<forward>)), METH_FASTCALL, nullptr},
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<norm>)), METH_FASTCALL, nullptr},
    {"lora", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<lora>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_torch() { return PyModule_Create(&module); }
