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
#include <vector>

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

// Tensors as a tuple.
PyObject *tuple_of(std::initializer_list<at::Tensor> tensors)
{
    PyObject *t = PyTuple_New((Py_ssize_t)tensors.size());
    Py_ssize_t i = 0;
    for (const at::Tensor &x : tensors) {
        PyObject *o = t ? THPVariable_Wrap(x) : nullptr;
        if (!o) {
            Py_XDECREF(t);
            return nullptr;
        }
        PyTuple_SET_ITEM(t, i++, o);
    }
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

// An activation tensor beside x: its type and shape.
Rows rows_like(PyObject *o, const at::Tensor &x, const char *name, int device)
{
    const at::Tensor &t = tensor(o, name);
    has_type(t, x.scalar_type(), name);
    if (t.sizes() != x.sizes())
        wrong_value(std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " + shape_text(x.sizes()));
    return rows_of(t, name, device);
}

// (x, gamma, eps, residual, quantise, return_y, return_rstd, y, q, total, stream) -> the outputs asked for, in the order
// y, or q and scale; total, with a residual; y, beside q; rstd.  One alone comes as it is.
PyObject *rms_norm(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    return guarded(count, 11, [&]() -> PyObject * {
        const at::Tensor &x = tensor(arg[0], "x");
        const int device = first_device(x, "x"), type = activation_type(x, "x");
        const Rows r = rows_of(x, "x", device);
        const float *gamma = vector_of(arg[1], r.c, "gamma", device);
        const double eps = PyFloat_AsDouble(arg[2]);
        if (eps == -1.0 && PyErr_Occurred()) return nullptr;
        const int quantise = PyObject_IsTrue(arg[4]), with_y = PyObject_IsTrue(arg[5]), with_rstd = PyObject_IsTrue(arg[6]);
        if (quantise < 0 || with_y < 0 || with_rstd < 0) return nullptr;
        const bool adds = arg[3] != Py_None, writes_y = !quantise || with_y || arg[7] != Py_None;
        Rows res{nullptr, 0, 0, 0}, rt{nullptr, 0, 0, 0}, ry{nullptr, 0, 0, 0}, rq{nullptr, 0, 0, 0};
        if (adds) res = rows_like(arg[3], x, "residual", device);
        if (!adds && arg[9] != Py_None) wrong_value("total is an output of calls with a residual");
        const Stream stream(arg[10], device);
        at::Tensor total, y, q, scale, rstd;
        if (adds) {
            total = output(arg[9], x.sizes(), x.scalar_type(), "total", stream);
            rt = rows_of(total, "total", device);
        }
        if (writes_y) {
            y = output(arg[7], x.sizes(), x.scalar_type(), "y", stream);
            ry = rows_of(y, "y", device);
        }
        const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
        if (quantise) {
            q = output(arg[8], x.sizes(), at::kChar, "q", stream);
            rq = rows_of(q, "q", device);
            scale = stream.empty(lead, at::kFloat);
        }
        if (with_rstd) rstd = stream.empty(lead, at::kFloat);
        if (r.rows) {
            float *rstd_at = with_rstd ? rstd.data_ptr<float>() : nullptr;
            check(quantise ? conv_bn_silu_rms_norm_quantize(r.data, r.distance, res.data, res.distance, gamma, (float)eps,
                                                            rt.data, rt.distance, ry.data, ry.distance, rq.data, rq.distance,
                                                            scale.data_ptr<float>(), rstd_at, r.rows, (int)r.c, type,
                                                            stream.handle)
                           : conv_bn_silu_rms_norm(r.data, r.distance, res.data, res.distance, gamma, (float)eps, rt.data,
                                                   rt.distance, ry.data, ry.distance, rstd_at, r.rows, (int)r.c, type,
                                                   stream.handle));
        }
        at::Tensor out[5];
        int n = 0;
        if (quantise) {
            out[n++] = q;
            out[n++] = scale;
        } else {
            out[n++] = y;
        }
        if (adds) out[n++] = total;
        if (quantise && writes_y) out[n++] = y;
        if (with_rstd) out[n++] = rstd;
        switch (n) {
        case 1: return THPVariable_Wrap(out[0]);
        case 2: return tuple_of({out[0], out[1]});
        case 3: return tuple_of({out[0], out[1], out[2]});
        case 4: return tuple_of({out[0], out[1], out[2], out[3]});
        default: return tuple_of({out[0], out[1], out[2], out[3], out[4]});
        }
    });
}

// (dy, x, gamma, rstd, residual, dx, stream) -> (dx, dgamma)
PyObject *rms_norm_backward(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    return guarded(count, 7, [&]() -> PyObject * {
        const at::Tensor &x = tensor(arg[1], "x");
        const int device = first_device(x, "x"), type = activation_type(x, "x");
        const Rows r = rows_of(x, "x", device), rdy = rows_like(arg[0], x, "dy", device);
        const float *gamma = vector_of(arg[2], r.c, "gamma", device);
        const float *rstd = vector_of(arg[3], r.rows, "rstd", device);
        if (!rstd && arg[3] == Py_None) wrong_type("rstd must be a torch.Tensor");
        Rows res{nullptr, 0, 0, 0};
        if (arg[4] != Py_None) res = rows_like(arg[4], x, "residual", device);
        const long long need = conv_bn_silu_rms_norm_backward_workspace(r.rows, (int)r.c);
        if (need < 0) throw Status{CBS_ERR_INVALID_ARG};
        const Stream stream(arg[6], device);
        const at::Tensor dx = output(arg[5], x.sizes(), x.scalar_type(), "dx", stream);
        const Rows rdx = rows_of(dx, "dx", device);
        const at::Tensor dgamma = stream.empty({r.c}, at::kFloat);
        const at::Tensor work = stream.empty({need}, at::kByte);
        check(conv_bn_silu_rms_norm_backward(rdy.data, rdy.distance, r.data, r.distance, gamma, rstd, res.data, res.distance,
                                             rdx.data, rdx.distance, dgamma.data_ptr<float>(), r.rows, (int)r.c, type,
                                             work.data_ptr(), need, stream.handle));
        return pair(dx, dgamma);
    });
}

// What both calls of the adapters share: x, index, a, b and scale.
struct Adapters {
    Rows x;
    const int *index;
    const void *a, *b;
    const float *scale;
    long long m, k, n, rank, adapters;
    int type;
    Adapters(PyObject *px, PyObject *pindex, PyObject *pa, PyObject *pb, PyObject *pscale, int device)
    {
        const at::Tensor &tx = tensor(px, "x"), &ti = tensor(pindex, "index"), &ta = tensor(pa, "a"), &tb = tensor(pb, "b");
        type = activation_type(tx, "x");
        x = rows_of(tx, "x", device);
        m = x.rows;
        k = x.c;
        has_type(ti, at::kInt, "index");
        if (!ti.is_cuda() || ti.get_device() != device || ti.numel() != m || !ti.is_contiguous())
            wrong_value("index must hold " + std::to_string(m) + " dense elements on the CUDA device of the call's first tensor");
        has_type(ta, tx.scalar_type(), "a");
        has_type(tb, tx.scalar_type(), "b");
        same_device(ta, "a", device);
        same_device(tb, "b", device);
        if (ta.dim() != 3 || ta.size(2) != k) wrong_value("a must be [adapters, rank, " + std::to_string(k) + "], got " + shape_text(ta.sizes()));
        adapters = ta.size(0);
        rank = ta.size(1);
        if (tb.dim() != 3 || tb.size(0) != adapters || tb.size(2) != rank)
            wrong_value("b must be [" + std::to_string(adapters) + ", n, " + std::to_string(rank) + "], got " + shape_text(tb.sizes()));
        n = tb.size(1);
        if (!ta.is_contiguous() || !tb.is_contiguous()) wrong_value("a and b must be dense");
        if (n > INT32_MAX || rank > INT32_MAX || adapters > INT32_MAX) throw Status{CBS_ERR_INVALID_ARG};
        index = ti.const_data_ptr<int>();
        a = ta.const_data_ptr();
        b = tb.const_data_ptr();
        scale = vector_of(pscale, adapters, "scale", device);
    }
};

// A tensor of x's type and the given shape.
Rows rows_shaped(PyObject *o, at::ScalarType type, at::IntArrayRef shape, const char *name, int device)
{
    const at::Tensor &t = tensor(o, name);
    has_type(t, type, name);
    if (t.sizes() != shape)
        wrong_value(std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
    return rows_of(t, name, device);
}

// (x, index, a, b, scale, base, return_hidden, y, stream) -> y or (y, hidden)
PyObject *linear_adapters(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    return guarded(count, 9, [&]() -> PyObject * {
        const at::Tensor &x = tensor(arg[0], "x");
        const int device = first_device(x, "x");
        const Adapters p(arg[0], arg[1], arg[2], arg[3], arg[4], device);
        const int with_hidden = PyObject_IsTrue(arg[6]);
        if (with_hidden < 0) return nullptr;
        c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
        shape.back() = p.n;
        Rows base{nullptr, 0, 0, 0};
        if (arg[5] != Py_None) base = rows_shaped(arg[5], x.scalar_type(), shape, "base", device);
        const long long need = conv_bn_silu_linear_adapters_workspace(p.m, (int)p.k, (int)p.n, (int)p.rank, (int)p.adapters);
        if (need < 0) throw Status{CBS_ERR_INVALID_ARG};
        const Stream stream(arg[8], device);
        const at::Tensor y = output(arg[7], shape, x.scalar_type(), "y", stream);
        const Rows ry = rows_of(y, "y", device);
        at::Tensor hidden, work;
        if (with_hidden) {
            shape.back() = p.rank;
            hidden = stream.empty(shape, at::kFloat);
        }
        if (need) work = stream.empty({need}, at::kByte);
        check(conv_bn_silu_linear_adapters(p.x.data, p.x.distance, p.index, p.a, p.b, p.scale, base.data, base.distance,
                                           ry.data, ry.distance, with_hidden ? hidden.data_ptr<float>() : nullptr, p.m,
                                           (int)p.k, (int)p.n, (int)p.rank, (int)p.adapters, p.type,
                                           need ? work.data_ptr() : nullptr, need, stream.handle));
        return with_hidden ? pair(y, hidden) : THPVariable_Wrap(y);
    });
}

// (dy, x, index, a, b, scale, hidden, base, dx, stream) -> (dx, da, db)
PyObject *linear_adapters_backward(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    return guarded(count, 10, [&]() -> PyObject * {
        const at::Tensor &x = tensor(arg[1], "x");
        const int device = first_device(x, "x");
        const Adapters p(arg[1], arg[2], arg[3], arg[4], arg[5], device);
        c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
        shape.back() = p.n;
        const Rows dy = rows_shaped(arg[0], x.scalar_type(), shape, "dy", device);
        const float *hidden = vector_of(arg[6], p.m * p.rank, "hidden", device);
        if (!hidden && arg[6] == Py_None) wrong_type("hidden must be a torch.Tensor");
        Rows base{nullptr, 0, 0, 0};
        if (arg[7] != Py_None) base = rows_shaped(arg[7], x.scalar_type(), x.sizes(), "base", device);
        const long long need =
            conv_bn_silu_linear_adapters_backward_workspace(p.m, (int)p.k, (int)p.n, (int)p.rank, (int)p.adapters);
        if (need < 0) throw Status{CBS_ERR_INVALID_ARG};
        const Stream stream(arg[9], device);
        const at::Tensor dx = output(arg[8], x.sizes(), x.scalar_type(), "dx", stream);
        const Rows rdx = rows_of(dx, "dx", device);
        const at::Tensor da = stream.empty({p.adapters, p.rank, p.k}, at::kFloat);
        const at::Tensor db = stream.empty({p.adapters, p.n, p.rank}, at::kFloat);
        const at::Tensor work = stream.empty({need}, at::kByte);
        check(conv_bn_silu_linear_adapters_backward(dy.data, dy.distance, p.x.data, p.x.distance, p.index, p.a, p.b, p.scale,
                                                    hidden, base.data, base.distance, rdx.data, rdx.distance,
                                                    da.data_ptr<float>(), db.data_ptr<float>(), p.m, (int)p.k, (int)p.n,
                                                    (int)p.rank, (int)p.adapters, p.type, work.data_ptr(), need,
                                                    stream.handle));
        return tuple_of({dx, da, db});
    });
}

// A list or tuple of tensors.
struct Tensors {
    PyObject *fast = nullptr;
    const char *name;
    Tensors(PyObject *o, const char *name) : name(name)
    {
        if (!PyList_Check(o) && !PyTuple_Check(o)) wrong_type(std::string(name) + " must be a list or tuple of tensors");
        fast = o;
    }
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
    const at::Tensor &at(Py_ssize_t i) const { return tensor(PySequence_Fast_GET_ITEM(fast, i), name); }
};

[[noreturn]] void wrong_item(const char *name, Py_ssize_t i, const std::string &what)
{
    wrong_value(std::string(name) + "[" + std::to_string(i) + "] " + what);
}

// A number, or a CUDA tensor of one element of `type` that the step reads on the device: its address.
const void *number_at(PyObject *o, at::ScalarType type, const char *name, int device)
{
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    has_type(t, type, name);
    if (!t.is_cuda() || t.get_device() != device || t.numel() != 1)
        wrong_value(std::string(name) + " must be a number or hold one element on the CUDA device of the call's first tensor");
    return t.const_data_ptr();
}

// (params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, step, lr, beta1, beta2, eps, weight_decay,
// grad_scale, stream) -> None; the scales both None for 32-bit moments
PyObject *adamw_step(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    return guarded(count, 14, [&]() -> PyObject * {
        const Tensors p(arg[0], "params"), g(arg[1], "grads"), m(arg[2], "exp_avg"), v(arg[3], "exp_avg_sq");
        const bool eight = arg[4] != Py_None || arg[5] != Py_None;
        const Tensors ms(eight ? arg[4] : arg[2], "exp_avg_scale"), vs(eight ? arg[5] : arg[2], "exp_avg_sq_scale");
        const Py_ssize_t n = p.size();
        for (const Tensors *t : {&g, &m, &v, &ms, &vs})
            if (t->size() != n)
                wrong_value(std::string(t->name) + " has " + std::to_string(t->size()) + " tensors, expected " + std::to_string(n));
        if (!n) Py_RETURN_NONE;
        const int device = first_device(p.at(0), "params[0]");
        const at::ScalarType state = eight ? at::kFloat8_e4m3fn : at::kFloat;
        auto dense = [&](const Tensors &t, Py_ssize_t i, int64_t elements) -> const at::Tensor & {
            const at::Tensor &x = t.at(i);
            if (!x.is_cuda() || x.get_device() != device) wrong_item(t.name, i, "must be on the CUDA device of the call's first tensor");
            if (x.numel() != elements) wrong_item(t.name, i, "has " + std::to_string(x.numel()) + " elements, expected " + std::to_string(elements));
            if (!x.is_contiguous()) wrong_item(t.name, i, "must be dense");
            return x;
        };
        std::vector<cbs_adamw_tensor> all((size_t)n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            cbs_adamw_tensor &e = all[(size_t)i];
            const int64_t elements = p.at(i).numel();
            const at::Tensor &tp = dense(p, i, elements), &tg = dense(g, i, elements), &tm = dense(m, i, elements),
                             &tv = dense(v, i, elements);
            e.param_dtype = activation_type(tp, "params");
            e.grad_dtype = activation_type(tg, "grads");
            has_type(tm, state, "exp_avg");
            has_type(tv, state, "exp_avg_sq");
            e.param = tp.data_ptr();
            e.grad = tg.data_ptr();
            e.exp_avg = tm.data_ptr();
            e.exp_avg_sq = tv.data_ptr();
            e.exp_avg_scale = e.exp_avg_sq_scale = nullptr;
            if (eight) {
                const at::Tensor &a = dense(ms, i, (elements + 255) / 256), &b = dense(vs, i, (elements + 255) / 256);
                has_type(a, at::kFloat, "exp_avg_scale");
                has_type(b, at::kFloat, "exp_avg_sq_scale");
                e.exp_avg_scale = static_cast<float *>(a.data_ptr());
                e.exp_avg_sq_scale = static_cast<float *>(b.data_ptr());
            }
            e.n = elements;
        }
        cbs_adamw_options o{};
        o.step_device = static_cast<const long long *>(number_at(arg[6], at::kLong, "step", device));
        o.lr_device = static_cast<const float *>(number_at(arg[7], at::kFloat, "lr", device));
        o.grad_scale_device = static_cast<const float *>(number_at(arg[12], at::kFloat, "grad_scale", device));
        if (!o.step_device) {
            o.step = PyLong_AsLongLong(arg[6]);
            if (o.step == -1 && PyErr_Occurred()) return nullptr;
        }
        double *const to[] = {&o.lr, &o.beta1, &o.beta2, &o.eps, &o.weight_decay, &o.grad_scale};
        for (int i = 0; i < 6; ++i) {
            PyObject *from = arg[7 + i];
            if ((i == 0 && o.lr_device) || (i == 5 && o.grad_scale_device)) continue;
            *to[i] = PyFloat_AsDouble(from);
            if (*to[i] == -1.0 && PyErr_Occurred()) return nullptr;
        }
        o.state_bits = eight ? 8 : 32;
        const Stream stream(arg[13], device);
        check(conv_bn_silu_adamw_step(all.data(), (int)n, &o, stream.handle));
        Py_RETURN_NONE;
    });
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {CALL(layer_norm), CALL(layer_norm_backward), CALL(quantize_rows), CALL(layer_norm_quantize),
                           CALL(linear_int8), CALL(rms_norm), CALL(rms_norm_backward), CALL(linear_adapters),
                           CALL(linear_adapters_backward), CALL(adamw_step),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_token_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__token_ops() { return PyModule_Create(&g_module); }
