// Python binding of the training operators (gated_act_training.h) against
// PyTorch's C++ interface: argument checks, output allocation and one call of
// the C ABI each.  training.py holds the documented functions, which hand
// their arguments on in order.
//
// Why not ctypes here: these calls allocate two to five tensors and launch one
// or two kernels of a few microseconds.  Measured on the GB300's host, a
// forward and backward pass of silu_and_mul over 64 rows took 31 us through
// ctypes and torch.empty, of which the two C calls were 7.5 us.
#include <Python.h>

#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gated_act_training.h"

namespace {

using at::Tensor;

PyObject *g_checkpoint, *g_balance, *g_check;   // training.Checkpoint, .BalanceLoss, _check

struct Error {   // becomes a Python exception; an empty message: one is set already
    PyObject *type;
    std::string message;
};
[[noreturn]] void value_error(const std::string &m) { throw Error{PyExc_ValueError, m}; }
[[noreturn]] void type_error(const std::string &m) { throw Error{PyExc_TypeError, m}; }

// ---------------------------------------------------------------- arguments

const Tensor &tensor(PyObject *o, const char *what) {
    if (!THPVariable_Check(o))
        type_error(std::string(what) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Error{nullptr, ""};
    return v;
}

double real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Error{nullptr, ""};
    return v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Error{nullptr, ""};
    return v != 0;
}

void reachable(const Tensor &x, const char *what) {
    if (!x.is_cuda() && !x.is_pinned())
        value_error(std::string(what) + " must be a CUDA tensor or page-locked host memory "
                                        "(the library has no CPU path)");
}

int dtype_code(at::ScalarType t) {
    switch (t) {
    case at::kBFloat16: return GATED_ACT_BF16;
    case at::kHalf: return GATED_ACT_F16;
    case at::kFloat: return GATED_ACT_F32;
    default: return -1;
    }
}

// A 2-D tensor with contiguous columns.
struct Rows {
    const Tensor &x;
    int64_t m, n, stride;
    int code;
    Rows(PyObject *o, const char *what) : x(tensor(o, what)) {
        if (x.dim() != 2)
            value_error(std::string(what) + " must be 2-D");
        code = dtype_code(x.scalar_type());
        if (code < 0)
            type_error(std::string(what) + " must be bfloat16, float16 or float32");
        reachable(x, what);
        m = x.size(0);
        n = x.size(1);
        if (x.stride(1) != 1 && n > 1)
            value_error(std::string(what) + ": columns must be contiguous");
        stride = m > 1 ? x.stride(0) : n;
    }
    void *data() const { return x.data_ptr(); }
};

// The address of a contiguous tensor of that type and shape.
void *flat(const Tensor &x, const char *what, at::ScalarType type, at::IntArrayRef shape) {
    if (x.scalar_type() != type || x.sizes() != shape || !x.is_contiguous()) {
        std::string s;
        for (const int64_t n : shape)
            s += (s.empty() ? "" : ", ") + std::to_string(n);
        value_error(std::string(what) + " must be a contiguous " + c10::toString(type) +
                    " tensor of shape [" + s + "]");
    }
    reachable(x, what);
    return x.data_ptr();
}

// The live row count, or null.
const int32_t *count(PyObject *o) {
    if (o == Py_None)
        return nullptr;
    const Tensor &x = tensor(o, "n_rows");
    if (x.scalar_type() != at::kInt || x.numel() < 1)
        value_error("n_rows must be an int32 tensor");
    reachable(x, "n_rows");
    return static_cast<const int32_t *>(x.data_ptr());
}

// ------------------------------------------------------ streams and outputs

// The stream of a call; what is allocated meanwhile belongs to it.
struct Launch {
    const Tensor &like;
    cudaStream_t stream;
    c10::cuda::OptionalCUDAStreamGuard guard;
    Launch(PyObject *o, const Tensor &like_) : like(like_) {
        const c10::DeviceIndex device =
            like.is_cuda() ? like.device().index() : c10::cuda::current_device();
        if (o == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(device).stream();
            return;
        }
        PyObject *handle = PyObject_GetAttrString(o, "cuda_stream");
        if (!handle)
            throw Error{nullptr, ""};
        void *p = PyLong_AsVoidPtr(handle);
        Py_DECREF(handle);
        if (PyErr_Occurred())
            throw Error{nullptr, ""};
        stream = static_cast<cudaStream_t>(p);
        guard.reset_stream(c10::cuda::getStreamFromExternal(stream, device));
    }
    // An uninitialised tensor where `like` lives.
    Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        if (!like.is_cuda())
            return at::empty(shape, at::TensorOptions().dtype(type).pinned_memory(true));
        return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
    }
    // Device memory for this call.
    Tensor scratch(size_t bytes) const {
        const at::Device device =
            like.is_cuda() ? like.device() : at::Device(at::kCUDA, c10::cuda::current_device());
        return Tensor(at::detail::empty_cuda({static_cast<int64_t>(bytes)}, at::kByte, device,
                                             std::nullopt));
    }
    Tensor output(PyObject *o, at::IntArrayRef shape, at::ScalarType type) const {
        if (o == Py_None)
            return empty(shape, type);
        const Tensor &x = tensor(o, "out");
        flat(x, "out", type, shape);
        return x;
    }
};

// Raises what gated_activation_gb300._check raises for a status other than 0.
void check(const char *fn, int rc) {
    if (rc == GATED_ACT_OK)
        return;
    PyObject *r = PyObject_CallFunction(g_check, "si", fn, rc);
    Py_XDECREF(r);
    if (r)
        PyErr_SetString(PyExc_RuntimeError, "status without an exception");
    throw Error{nullptr, ""};
}

PyObject *wrap(const Tensor &x) { return THPVariable_Wrap(x); }
PyObject *none() { return Py_NewRef(Py_None); }

// A tuple of new references, or an instance of the named tuple `cls` of them.
template <class... A> PyObject *pack(PyObject *cls, A... a) {
    PyObject *items[] = {a...};
    constexpr Py_ssize_t n = sizeof...(A);
    PyObject *t = PyTuple_New(n);
    for (Py_ssize_t i = 0; i < n; ++i)
        if (t)
            PyTuple_SET_ITEM(t, i, items[i]);
        else
            Py_XDECREF(items[i]);
    if (!t || !cls)
        return t;
    PyObject *args = PyTuple_Pack(1, t);
    Py_DECREF(t);
    if (!args)
        return nullptr;
    PyObject *r = PyTuple_Type.tp_new(reinterpret_cast<PyTypeObject *>(cls), args, nullptr);
    Py_DECREF(args);
    return r;
}

template <class T> T *ptr(const Tensor &x) { return static_cast<T *>(x.data_ptr()); }

// --------------------------------------------------------------- checkpoints

int64_t gated_width(const Rows &x, PyObject *d_) {
    int64_t d = x.n / 2;
    if (d_ != Py_None)
        d = integer(d_);
    else if (x.n % 2)
        value_error("odd row length: pass d explicitly");
    if (d < 1 || d > x.n / 2)
        value_error("rows are shorter than 2d");
    return d;
}

// (x, n_rows, d, out, stream)
template <class F> PyObject *checkpoint(const char *fn, F f, PyObject *const *a) {
    const Rows x(a[0], "input");
    const int64_t d = gated_width(x, a[2]);
    const int32_t *n_rows = count(a[1]);
    const Launch go(a[4], x.x);
    const Tensor out = go.output(a[3], {x.m, d}, x.x.scalar_type());
    const Tensor codes = go.empty({x.m, 2 * d}, at::kChar);
    const Tensor scales = go.empty({x.m, gated_act_checkpoint_scales(d)}, at::kByte);
    check(fn, f(out.data_ptr(), ptr<int8_t>(codes), ptr<uint8_t>(scales), x.data(), x.m, d,
                x.stride, x.code, n_rows, go.stream));
    return pack(nullptr, wrap(out), pack(g_checkpoint, wrap(codes), wrap(scales), none()));
}
PyObject *silu_checkpoint(PyObject *const *a) {
    return checkpoint("silu_and_mul_checkpoint", silu_and_mul_checkpoint, a);
}
PyObject *gelu_checkpoint(PyObject *const *a) {
    return checkpoint("gelu_and_mul_checkpoint", gelu_and_mul_checkpoint, a);
}

// (x, z, d, out, stream)
PyObject *sparse_checkpoint(PyObject *const *a) {
    const Rows x(a[0], "input");
    const double z = real(a[1]);
    const int64_t d = gated_width(x, a[2]);
    const Launch go(a[4], x.x);
    const Tensor out = go.output(a[3], {x.m, d}, x.x.scalar_type());
    const Tensor codes = go.empty({x.m, 2 * d}, at::kChar);
    const Tensor scales = go.empty({x.m, gated_act_checkpoint_scales(d)}, at::kByte);
    const Tensor std = go.empty({x.m}, at::kFloat);
    check("gelu_and_mul_sparse_checkpoint",
          gelu_and_mul_sparse_checkpoint(out.data_ptr(), ptr<int8_t>(codes), ptr<uint8_t>(scales),
                                         ptr<float>(std), x.data(), x.m, d, x.stride, z, x.code,
                                         go.stream));
    return pack(nullptr, wrap(out), pack(g_checkpoint, wrap(codes), wrap(scales), wrap(std)));
}

// codes and scales of a checkpoint of rows [m, 2d]
struct Kept {
    const int8_t *codes;
    const uint8_t *scales;
    PyObject *std;
    const Tensor &x;
    Kept(PyObject *o) : std(nullptr), x(tensor(item(o, 0), "codes")) {}
    static PyObject *item(PyObject *o, Py_ssize_t i) {
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3)
            type_error("the second argument must be a Checkpoint");
        return PyTuple_GET_ITEM(o, i);
    }
    void expect(PyObject *o, int64_t m, int64_t d) {
        codes = static_cast<const int8_t *>(flat(x, "codes", at::kChar, {m, 2 * d}));
        scales = static_cast<const uint8_t *>(
            flat(tensor(item(o, 1), "scales"), "scales", at::kByte, {m, gated_act_checkpoint_scales(d)}));
        std = item(o, 2);
    }
};

PyObject *gradients(const Tensor &grad_in, const Tensor &out) {
    return out.defined() ? pack(nullptr, wrap(grad_in), wrap(out)) : wrap(grad_in);
}

// (grad_out, kept, n_rows, recompute, stream)
template <class F> PyObject *backward(const char *fn, F f, PyObject *const *a) {
    const Rows g(a[0], "grad_out");
    Kept kept(a[1]);
    kept.expect(a[1], g.m, g.n);
    const int32_t *n_rows = count(a[2]);
    const Launch go(a[4], g.x);
    const at::ScalarType type = g.x.scalar_type();
    const Tensor grad_in = go.empty({g.m, 2 * g.n}, type);
    const Tensor out = truth(a[3]) ? go.empty({g.m, g.n}, type) : Tensor();
    check(fn, f(grad_in.data_ptr(), out.defined() ? out.data_ptr() : nullptr, g.data(), kept.codes,
                kept.scales, g.m, g.n, g.stride, g.code, n_rows, go.stream));
    return gradients(grad_in, out);
}
PyObject *silu_backward(PyObject *const *a) {
    return backward("silu_and_mul_backward", silu_and_mul_backward, a);
}
PyObject *gelu_backward(PyObject *const *a) {
    return backward("gelu_and_mul_backward", gelu_and_mul_backward, a);
}

// (grad_out, kept, z, recompute, stream)
PyObject *sparse_backward(PyObject *const *a) {
    const Rows g(a[0], "grad_out");
    Kept kept(a[1]);
    kept.expect(a[1], g.m, g.n);
    if (kept.std == Py_None)
        value_error("the checkpoint of gelu_and_mul_sparse holds std");
    const float *std =
        static_cast<const float *>(flat(tensor(kept.std, "std"), "std", at::kFloat, {g.m}));
    const double z = real(a[2]);
    const Launch go(a[4], g.x);
    const at::ScalarType type = g.x.scalar_type();
    const Tensor grad_in = go.empty({g.m, 2 * g.n}, type);
    const Tensor out = truth(a[3]) ? go.empty({g.m, g.n}, type) : Tensor();
    check("gelu_and_mul_sparse_backward",
          gelu_and_mul_sparse_backward(grad_in.data_ptr(), out.defined() ? out.data_ptr() : nullptr,
                                       g.data(), kept.codes, kept.scales, std, g.m, g.n, g.stride,
                                       z, g.code, go.stream));
    return gradients(grad_in, out);
}

// (kept, fp32, stream)
PyObject *values(PyObject *const *a) {
    Kept kept(a[0]);
    if (kept.x.dim() != 2 || kept.x.size(1) % 2 || kept.x.size(1) < 2)
        value_error("codes must be 2-D [M, 2d]");
    const int64_t m = kept.x.size(0), d = kept.x.size(1) / 2;
    kept.expect(a[0], m, d);
    const bool wide = truth(a[1]);
    const Launch go(a[2], kept.x);
    const Tensor v = go.empty({m, 2 * d}, wide ? at::kFloat : at::kBFloat16);
    check("gated_act_checkpoint_values",
          gated_act_checkpoint_values(v.data_ptr(), kept.codes, kept.scales, m, d,
                                      wide ? GATED_ACT_F32 : GATED_ACT_BF16, go.stream));
    return wrap(v);
}

// ---------------------------------------------------------------- layer norm

const void *parameter(PyObject *o, const char *what, at::ScalarType type, int64_t d) {
    return o == Py_None ? nullptr : flat(tensor(o, what), what, type, {d});
}

at::ScalarType parameter_type(PyObject *weight, const Rows &x) {
    const at::ScalarType t = tensor(weight, "weight").scalar_type();
    if (t != x.x.scalar_type() && t != at::kFloat)
        type_error("weight must have the input's type or be float32");
    return t;
}

// (x, weight, bias, eps, out, stream)
PyObject *norm(PyObject *const *a) {
    const Rows x(a[0], "input");
    const at::ScalarType wt = parameter_type(a[1], x);
    const void *w = parameter(a[1], "weight", wt, x.n), *b = parameter(a[2], "bias", wt, x.n);
    const double eps = real(a[3]);
    const Launch go(a[5], x.x);
    const Tensor out = go.output(a[4], {x.m, x.n}, x.x.scalar_type());
    const Tensor mean = go.empty({x.m}, at::kFloat), rstd = go.empty({x.m}, at::kFloat);
    check("layer_norm", layer_norm(out.data_ptr(), ptr<float>(mean), ptr<float>(rstd), x.data(), w,
                                   b, x.m, x.n, x.stride, eps, x.code, dtype_code(wt), go.stream));
    return pack(nullptr, wrap(out), wrap(mean), wrap(rstd));
}

// (grad_out, x, weight, mean, rstd, bias, stream)
PyObject *norm_backward(PyObject *const *a) {
    const Rows g(a[0], "grad_out"), x(a[1], "input");
    if (g.m != x.m || g.n != x.n || g.code != x.code)
        value_error("grad_out must have the shape and type of the input");
    const at::ScalarType wt = parameter_type(a[2], x);
    const void *w = parameter(a[2], "weight", wt, x.n);
    const float *mean =
        static_cast<const float *>(flat(tensor(a[3], "mean"), "mean", at::kFloat, {x.m}));
    const float *rstd =
        static_cast<const float *>(flat(tensor(a[4], "rstd"), "rstd", at::kFloat, {x.m}));
    const bool bias = truth(a[5]);
    const Launch go(a[6], x.x);
    const Tensor grad_in = go.empty({x.m, x.n}, x.x.scalar_type());
    const Tensor gw = go.empty({x.n}, at::kFloat);
    const Tensor gb = bias ? go.empty({x.n}, at::kFloat) : Tensor();
    const size_t need = layer_norm_backward_workspace_bytes(x.m, x.n);
    const Tensor ws = go.scratch(need);
    check("layer_norm_backward",
          layer_norm_backward(grad_in.data_ptr(), ptr<float>(gw), bias ? ptr<float>(gb) : nullptr,
                              g.data(), x.data(), w, mean, rstd, x.m, x.n, x.stride, g.stride,
                              x.code, dtype_code(wt), ws.data_ptr(), need, go.stream));
    return pack(nullptr, wrap(grad_in), wrap(gw), bias ? wrap(gb) : none());
}

// -------------------------------------------------------------- balance loss

const uint8_t *live_tokens(PyObject *o, int64_t t) {
    if (o == Py_None)
        return nullptr;
    const Tensor &x = tensor(o, "live");
    if (x.scalar_type() != at::kBool && x.scalar_type() != at::kByte)
        type_error("live must be bool or uint8");
    return static_cast<const uint8_t *>(flat(x, "live", x.scalar_type(), {t}));
}

// (logits, ids, coef, live, stream)
PyObject *balance(PyObject *const *a) {
    const Rows x(a[0], "logits");
    const Tensor &ids = tensor(a[1], "ids");
    const at::ScalarType it = ids.scalar_type();
    if (ids.dim() != 2 || ids.size(0) != x.m || (it != at::kInt && it != at::kLong))
        value_error("ids must be [T, k] int32 or int64");
    const int64_t k = ids.size(1);
    const void *chosen = flat(ids, "ids", it, {x.m, k});
    const double coef = real(a[2]);
    const uint8_t *live = live_tokens(a[3], x.m);
    const Launch go(a[4], x.x);
    const Tensor loss = go.empty({1}, at::kFloat), mean_p = go.empty({x.n}, at::kFloat);
    const Tensor tokens = go.empty({1}, at::kInt), counts = go.empty({x.n}, at::kInt);
    const size_t need = moe_balance_loss_workspace_bytes(x.m, x.n);
    const Tensor ws = go.scratch(need);
    check("moe_balance_loss",
          moe_balance_loss(ptr<float>(loss), ptr<int32_t>(counts), ptr<int32_t>(tokens),
                           ptr<float>(mean_p), x.data(), chosen, live, x.m, x.n, k, x.stride,
                           x.code, it == at::kLong, coef, ws.data_ptr(), need, go.stream));
    return pack(g_balance, wrap(loss), wrap(counts), wrap(tokens), wrap(mean_p),
                PyLong_FromLongLong(k), PyFloat_FromDouble(coef));
}

// (grad_loss, logits, kept, live, stream)
PyObject *balance_backward(PyObject *const *a) {
    const Tensor &grad_loss = tensor(a[0], "grad_loss");
    const Rows x(a[1], "logits");
    if (grad_loss.scalar_type() != at::kFloat || grad_loss.numel() != 1)
        value_error("grad_loss must be an fp32 tensor of one element");
    reachable(grad_loss, "grad_loss");
    if (!PyTuple_Check(a[2]) || PyTuple_GET_SIZE(a[2]) != 6)
        type_error("the third argument must be a BalanceLoss");
    const auto item = [&](Py_ssize_t i) { return PyTuple_GET_ITEM(a[2], i); };
    const void *counts = flat(tensor(item(1), "counts"), "counts", at::kInt, {x.n});
    const void *tokens = flat(tensor(item(2), "tokens"), "tokens", at::kInt, {1});
    const int64_t k = integer(item(4));
    const double coef = real(item(5));
    const uint8_t *live = live_tokens(a[3], x.m);
    const Launch go(a[4], x.x);
    const Tensor grad = go.empty({x.m, x.n}, x.x.scalar_type());
    check("moe_balance_loss_backward",
          moe_balance_loss_backward(grad.data_ptr(), ptr<const float>(grad_loss), x.data(),
                                    static_cast<const int32_t *>(counts),
                                    static_cast<const int32_t *>(tokens), live, x.m, x.n, k,
                                    x.stride, x.code, coef, go.stream));
    return wrap(grad);
}

// -------------------------------------------------------------------- module

// N positional arguments to f; C++ exceptions to Python's.
template <PyObject *(*f)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N)
        return PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    try {
        return f(args);
    } catch (const Error &e) {
        if (!e.message.empty())
            PyErr_SetString(e.type, e.message.c_str());
    } catch (const c10::OutOfMemoryError &e) {
        // the class that torch's own functions raise
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *cls = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (cls)
            PyErr_SetString(cls, e.what_without_backtrace());
        Py_XDECREF(cls);
        Py_XDECREF(torch);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (Checkpoint, BalanceLoss, check)
PyObject *set_up(PyObject *const *a) {
    g_checkpoint = Py_NewRef(a[0]);
    g_balance = Py_NewRef(a[1]);
    g_check = Py_NewRef(a[2]);
    return none();
}

#define ENTRY(name, f, n) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {
    ENTRY("set_up", set_up, 3),
    ENTRY("silu_and_mul_checkpoint", silu_checkpoint, 5),
    ENTRY("gelu_and_mul_checkpoint", gelu_checkpoint, 5),
    ENTRY("gelu_and_mul_sparse_checkpoint", sparse_checkpoint, 5),
    ENTRY("silu_and_mul_backward", silu_backward, 5),
    ENTRY("gelu_and_mul_backward", gelu_backward, 5),
    ENTRY("gelu_and_mul_sparse_backward", sparse_backward, 5),
    ENTRY("checkpoint_values", values, 3),
    ENTRY("layer_norm", norm, 6),
    ENTRY("layer_norm_backward", norm_backward, 7),
    ENTRY("moe_balance_loss", balance, 5),
    ENTRY("moe_balance_loss_backward", balance_backward, 5),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_training", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__training() { return PyModule_Create(&g_module); }
