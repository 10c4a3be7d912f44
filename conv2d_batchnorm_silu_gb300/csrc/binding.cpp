// binding.cpp -- the Python calls of the token-wise operators (conv_bn_silu.h), as a CPython module
// over PyTorch's C++ tensors.  Argument marshalling only: checks of devices, types and shapes, outputs
// and workspaces from PyTorch's allocator, the current stream.  It is compiled because these calls are
// often small and bound by the host: a layer norm of 1024x32 took 10.5 us through ctypes and Python on
// the GB300's host and takes half of that here.  capi.py holds the documented functions.
//
// A function returns its tensors, raises TypeError or ValueError, or returns the C library's status as
// an int when that is not CBS_OK.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <optional>
#include <string>

#include "conv_bn_silu.h"

namespace {

// A Python exception to raise.
struct Refused {
    PyObject *type;
    std::string text;
};
[[noreturn]] void wrong_type(const std::string &text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void wrong_value(const std::string &text) { throw Refused{PyExc_ValueError, text}; }

// A C library status to return.
struct Status {
    int code;
};
void check(int status)
{
    if (status != CBS_OK) throw Status{status};
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) wrong_type(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

// The device of a call's first tensor, which has to be the current one.
int first_device(const at::Tensor &t, const char *name)
{
    if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
        wrong_value(std::string(name) + " must be on the current CUDA device");
    return (int)t.get_device();
}

void same_device(const at::Tensor &t, const char *name, int device)
{
    if (!t.is_cuda() || t.get_device() != device)
        wrong_value(std::string(name) + " must be on the CUDA device of the call's first tensor");
}

void has_type(const at::Tensor &t, at::ScalarType type, const char *name)
{
    if (t.scalar_type() != type)
        wrong_type(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
}

int activation_type(const at::Tensor &t, const char *name)
{
    switch (t.scalar_type()) {
    case at::kFloat: return CBS_DTYPE_F32;
    case at::kBFloat16: return CBS_DTYPE_BF16;
    case at::kHalf: return CBS_DTYPE_F16;
    default:
        wrong_type(std::string(name) + " must be torch.float32, torch.bfloat16 or torch.float16, got " +
                   c10::toString(t.scalar_type()));
    }
}

// An activation tensor [..., c] as rows of c elements at one distance.
struct Rows {
    void *data;
    long long rows, distance;
    long long c;
};

Rows rows_of(const at::Tensor &t, const char *name, int device)
{
    same_device(t, name, device);
    const auto sizes = t.sizes(), strides = t.strides();
    const int64_t n = t.dim();
    if (n == 0) wrong_value(std::string(name) + " must have at least one dimension");
    Rows r{t.data_ptr(), 1, 0, sizes[n - 1]};
    if (r.c > 1 && strides[n - 1] != 1) wrong_value(std::string(name) + "'s last dimension must be dense");
    for (int64_t i = n - 2; i >= 0; --i) {
        if (sizes[i] == 1) continue;
        // Dimension i continues the rows that the inner dimensions gave.
        if (r.rows == 1)
            r.distance = strides[i];
        else if (sizes[i] > 1 && strides[i] != r.distance * r.rows && t.numel() != 0)
            wrong_value(std::string(name) + "'s leading dimensions must be rows at one distance");
        r.rows *= sizes[i];
    }
    if (r.rows <= 1) r.distance = r.c;
    if (r.c > INT32_MAX) throw Status{CBS_ERR_INVALID_ARG};
    return r;
}

const float *vector_of(PyObject *o, long long n, const char *name, int device)
{
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    has_type(t, at::kFloat, name);
    if (!t.is_cuda() || t.get_device() != device || t.numel() != n || !t.is_contiguous())
        wrong_value(std::string(name) + " must hold " + std::to_string(n) +
                    " dense elements on the CUDA device of the call's first tensor");
    return t.const_data_ptr<float>();
}

// The call's stream: the current one, or the one given, from whose memory outputs and workspaces come.
struct Stream {
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    cudaStream_t handle;
    int device;
    Stream(PyObject *o, int device) : device(device)
    {
        if (o != Py_None) {
            void *p = PyLong_AsVoidPtr(o);
            if (PyErr_Occurred()) {
                PyErr_Clear();
                wrong_type("stream must be a CUDA stream");
            }
            // The runtime's handle for the default stream, whose number PyTorch gives a stream of its own.
            if (p == static_cast<void *>(cudaStreamLegacy)) p = nullptr;
            guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), (c10::DeviceIndex)device));
        }
        handle = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const
    {
        return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt);
    }
};

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

// An output that is given or made here.
at::Tensor output(PyObject *o, at::IntArrayRef shape, at::ScalarType type, const char *name, const Stream &stream)
{
    if (o == Py_None) return stream.empty(shape, type);
    const at::Tensor &t = tensor(o, name);
    has_type(t, type, name);
    if (t.sizes() != shape)
        wrong_value(std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
    return t;
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b)
{
    PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b);
    PyObject *t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

// Runs a call and turns what it throws into what Python sees.
template <typename F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F &&f)
{
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", given, wanted);
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.text.c_str());
    } catch (const Status &s) {
        return PyLong_FromLong(s.code);
    } catch (...) {  // PyTorch's, as PyTorch raises them (torch.OutOfMemoryError and the others)
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// (x, gamma, beta, eps, return_stats, y, stream) -> y or (y, stats)
PyObject *layer_norm(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    return guarded(count, 7, [&]() -> PyObject * {
        const at::Tensor &x = tensor(arg[0], "x");
        const int device = first_device(x, "x"), type = activation_type(x, "x");
        const Rows r = rows_of(x, "x", device);
        const float *gamma = vector_of(arg[1], r.c, "gamma", device), *beta = vector_of(arg[2], r.c, "beta", device);
        const double eps = PyFloat_AsDouble(arg[3]);
        if (eps == -1.0 && PyErr_Occurred()) return nullptr;
        const int with_stats = PyObject_IsTrue(arg[4]);
        if (with_stats < 0) return nullptr;
        const Stream stream(arg[6], device);
        const at::Tensor y = output(arg[5], x.sizes(), x.scalar_type(), "y", stream);
        const Rows ry = rows_of(y, "y", device);
        at::Tensor stats;
        if (with_stats) stats = stream.empty({2, r.rows}, at::kFloat);
        if (r.rows)
            check(conv_bn_silu_layer_norm(r.data, r.distance, gamma, beta, (float)eps, ry.data, ry.distance,
                                          with_stats ? stats.data_ptr<float>() : nullptr, r.rows, (int)r.c, type,
                                          stream.handle));
        return with_stats ? pair(y, stats) : THPVariable_Wrap(y);
    });
}

// (dy, x, gamma, stats, dx, stream) -> (dx, dgamma, dbeta)
PyObject *layer_norm_backward(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    return guarded(count, 6, [&]() -> PyObject * {
        const at::Tensor &dy = tensor(arg[0], "dy"), &x = tensor(arg[1], "x");
        const int device = first_device(x, "x"), type = activation_type(x, "x");
        has_type(dy, x.scalar_type(), "dy");
        if (dy.sizes() != x.sizes())
            wrong_value("dy has shape " + shape_text(dy.sizes()) + ", expected " + shape_text(x.sizes()));
        const Rows r = rows_of(x, "x", device), rdy = rows_of(dy, "dy", device);
        const float *gamma = vector_of(arg[2], r.c, "gamma", device);
        const float *stats = vector_of(arg[3], 2 * r.rows, "stats", device);
        if (!stats) wrong_type("stats must be a torch.Tensor");
        const long long need = conv_bn_silu_layer_norm_backward_workspace(r.rows, (int)r.c);
        if (need < 0) throw Status{CBS_ERR_INVALID_ARG};
        const Stream stream(arg[5], device);
        const at::Tensor dx = output(arg[4], x.sizes(), x.scalar_type(), "dx", stream);
        const Rows rdx = rows_of(dx, "dx", device);
        const at::Tensor dgamma = stream.empty({r.c}, at::kFloat), dbeta = stream.empty({r.c}, at::kFloat);
        const at::Tensor work = stream.empty({need}, at::kByte);
        check(conv_bn_silu_layer_norm_backward(rdy.data, rdy.distance, r.data, r.distance, gamma, stats, rdx.data,
                                               rdx.distance, dgamma.data_ptr<float>(), dbeta.data_ptr<float>(), r.rows,
                                               (int)r.c, type, work.data_ptr(), need, stream.handle));
        PyObject *a = THPVariable_Wrap(dx), *b = THPVariable_Wrap(dgamma), *c = THPVariable_Wrap(dbeta);
        PyObject *t = a && b && c ? PyTuple_Pack(3, a, b, c) : nullptr;
        Py_XDECREF(a);
        Py_XDECREF(b);
        Py_XDECREF(c);
        return t;
    });
}

// Rows quantised, normalised before or not.
PyObject *quantise(PyObject *px, PyObject *pgamma, PyObject *pbeta, PyObject *peps, PyObject *pq, PyObject *pstream)
{
    const at::Tensor &x = tensor(px, "x");
    const int device = first_device(x, "x"), type = activation_type(x, "x");
    const Rows r = rows_of(x, "x", device);
    const float *gamma = pgamma ? vector_of(pgamma, r.c, "gamma", device) : nullptr;
    const float *beta = pbeta ? vector_of(pbeta, r.c, "beta", device) : nullptr;
    const double eps = peps ? PyFloat_AsDouble(peps) : 0.0;
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const Stream stream(pstream, device);
    const at::Tensor q = output(pq, x.sizes(), at::kChar, "q", stream);
    const Rows rq = rows_of(q, "q", device);
    const at::Tensor scale = stream.empty(x.sizes().slice(0, x.dim() - 1), at::kFloat);
    if (r.rows) {
        if (peps)
            check(conv_bn_silu_layer_norm_quantize(r.data, r.distance, gamma, beta, (float)eps, rq.data, rq.distance,
                                                   scale.data_ptr<float>(), r.rows, (int)r.c, type, stream.handle));
        else
            check(conv_bn_silu_quantize_rows(r.data, r.distance, rq.data, rq.distance, scale.data_ptr<float>(), r.rows,
                                             (int)r.c, type, stream.handle));
    }
    return pair(q, scale);
}

// (x, q, stream) -> (q, scale)
PyObject *quantize_rows(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    return guarded(count, 3, [&] { return quantise(arg[0], nullptr, nullptr, nullptr, arg[1], arg[2]); });
}

// (x, gamma, beta, eps, q, stream) -> (q, scale)
PyObject *layer_norm_quantize(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    return guarded(count, 6, [&] { return quantise(arg[0], arg[1], arg[2], arg[3], arg[4], arg[5]); });
}

// (a, w, a_scale, w_scale, bias, activation, residual, out_dtype, y, stream) -> y; activation a
// cbs_activation, out_dtype a cbs_dtype
PyObject *linear_int8(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    return guarded(count, 10, [&]() -> PyObject * {
        const at::Tensor &a = tensor(arg[0], "a"), &w = tensor(arg[1], "w");
        const int device = first_device(a, "a");
        has_type(a, at::kChar, "a");
        has_type(w, at::kChar, "w");
        if (w.dim() != 2) wrong_value("w must be [n, k]");
        const Rows rw = rows_of(w, "w", device), ra = rows_of(a, "a", device);
        if (ra.c != rw.c)
            wrong_value("channel mismatch: a has " + std::to_string(ra.c) + ", w has " + std::to_string(rw.c));
        const long long m = ra.rows, n = rw.rows, k = rw.c;
        const float *a_scale = vector_of(arg[2], m, "a_scale", device), *w_scale = vector_of(arg[3], n, "w_scale", device);
        if (!a_scale && m && arg[2] == Py_None) wrong_type("a_scale must be a torch.Tensor");
        if (!w_scale && n && arg[3] == Py_None) wrong_type("w_scale must be a torch.Tensor");
        const float *bias = vector_of(arg[4], n, "bias", device);
        const int activation = (int)PyLong_AsLong(arg[5]), out = (int)PyLong_AsLong(arg[7]);
        if (PyErr_Occurred()) return nullptr;
        const at::ScalarType type = out == CBS_DTYPE_F32 ? at::kFloat : (out == CBS_DTYPE_BF16 ? at::kBFloat16 : at::kHalf);
        c10::SmallVector<int64_t, 6> shape(a.sizes().begin(), a.sizes().end());
        shape.back() = n;
        Rows res{nullptr, 0, 0, 0};
        if (arg[6] != Py_None) {
            const at::Tensor &t = tensor(arg[6], "residual");
            has_type(t, type, "residual");
            if (t.sizes() != at::IntArrayRef(shape))
                wrong_value("residual has shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
            res = rows_of(t, "residual", device);
        }
        const Stream stream(arg[9], device);
        const at::Tensor y = output(arg[8], shape, type, "y", stream);
        if (m && n) {
            if (n > INT32_MAX) throw Status{CBS_ERR_INVALID_ARG};
            const Rows ry = rows_of(y, "y", device);
            const long long need = conv_bn_silu_linear_int8_workspace(m, (int)n, (int)k);
            if (need < 0) throw Status{CBS_ERR_INVALID_ARG};
            at::Tensor work;
            if (need) work = stream.empty({need}, at::kByte);
            check(conv_bn_silu_linear_int8(ra.data, ra.distance, rw.data, rw.distance, a_scale, w_scale, bias, res.data,
                                           res.distance, ry.data, ry.distance, m, (int)n, (int)k, activation, out,
                                           need ? work.data_ptr() : nullptr, need, stream.handle));
        }
        return THPVariable_Wrap(y);
    });
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {CALL(layer_norm), CALL(layer_norm_backward), CALL(quantize_rows), CALL(layer_norm_quantize),
                           CALL(linear_int8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_token_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__token_ops() { return PyModule_Create(&g_module); }
