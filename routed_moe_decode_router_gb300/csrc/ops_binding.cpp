// ops_binding.cpp -- the calls of ops.py as a CPython extension: it checks
// the tensors' attributes, allocates the outputs through PyTorch and calls
// the C ABI of include/moe_ops.h on the current stream.  It exists for the
// host's time: a call for one token is a few microseconds of GPU work, and
// marshalling it through Python and ctypes took 25.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "moe_ops.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refusal {
    PyObject *type;
    std::string text;
};
[[noreturn]] void value_error(const std::string &s) { throw Refusal{PyExc_ValueError, s}; }

PyObject *g_moe_error = nullptr;  // native.MoeError

struct Status {
    moe_status s;
};
void check(moe_status s) {
    if (s != MOE_OK) throw Status{s};
}

template <typename F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const Refusal &r) {
        PyErr_SetString(r.type, r.text.c_str());
    } catch (const Status &s) {
        PyObject *e = PyObject_CallFunction(g_moe_error, "is", (int)s.s, moe_last_error());
        if (e) {
            PyErr_SetObject(g_moe_error, e);
            Py_DECREF(e);
        }
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o))
        throw Refusal{PyExc_TypeError, std::string(name) + " must be a torch.Tensor"};
    return THPVariable_Unpack(o);
}

std::string text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

// The tensor that names the call's device: `dims` dimensions, in the current
// CUDA device's memory.
const Tensor &first(PyObject *o, const char *name, int64_t dims) {
    const Tensor &t = tensor(o, name);
    const auto n = [&] { return std::string(name); };
    if (t.dim() != dims)
        value_error(n() + " has " + std::to_string(t.dim()) + " dimensions, expected " +
                    std::to_string(dims));
    if (!t.is_cuda())
        value_error(n() + " is on " + t.device().str() + "; it must be in CUDA device memory");
    if (t.device().index() != c10::cuda::current_device())
        value_error(n() + " is on " + t.device().str() + ", which is not the current device");
    return t;
}

// Refuse what the kernels would misread.  strided: a row stride is taken, so
// only the last dimension has to be contiguous.
const Tensor &need(const Tensor &t, const char *name, ScalarType type, at::IntArrayRef shape,
                   const at::Device &dev, bool strided = false) {
    const auto n = [&] { return std::string(name); };
    if (t.scalar_type() != type)
        value_error(n() + " has dtype " + c10::toString(t.scalar_type()) + ", expected " +
                    c10::toString(type));
    if (t.sizes() != shape)
        value_error(n() + " has shape " + text(t.sizes()) + ", expected " + text(shape));
    if (!t.is_contiguous() && !(strided && t.dim() == 2 && t.stride(1) == 1))
        value_error(n() + " must be contiguous" + (strided ? " in its rows" : ""));
    if (t.device() != dev)
        value_error(n() + " is on " + t.device().str() + ", expected " + dev.str());
    return t;
}
const Tensor &need(PyObject *o, const char *name, ScalarType type, at::IntArrayRef shape,
                   const at::Device &dev, bool strided = false) {
    return need(tensor(o, name), name, type, shape, dev, strided);
}

int code_of(ScalarType t) {
    return t == at::kBFloat16 ? MOEOP_BF16 : t == at::kHalf ? MOEOP_FP16
           : t == at::kFloat  ? MOEOP_FP32 : -1;
}
ScalarType type_of(long code) {
    return code == MOEOP_BF16 ? at::kBFloat16 : code == MOEOP_FP16 ? at::kHalf : at::kFloat;
}
constexpr ScalarType kF8 = at::kFloat8_e4m3fn;

// The stride of a single row means nothing and may be anything.
int64_t row_stride(const Tensor &t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }
int64_t blocks(int64_t n) { return (n + MOEOP_BLOCK - 1) / MOEOP_BLOCK; }
int small(int64_t n, const char *name) {
    if (n > INT32_MAX || n < INT32_MIN) value_error(std::string(name) + " is out of range");
    return (int)n;
}
// From PyTorch's caching allocator, without the dispatcher's round trip.
Tensor fresh(at::IntArrayRef shape, ScalarType type, const at::Device &dev) {
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}
void *stream_of(const at::Device &dev) {
    return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
}
template <typename T>
T *ptr(const Tensor &t) {
    return static_cast<T *>(t.data_ptr());
}
PyObject *wrapped(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
bool counted(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return false;
}

// (x, weight, eps, residual, quantize, keep, residual_out)
PyObject *rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!counted(n, 7)) return nullptr;
    const double eps = PyFloat_AsDouble(a[2]);
    if (PyErr_Occurred()) return nullptr;
    return guarded([&] {
        const Tensor &x = first(a[0], "x", 2);
        const at::Device dev = x.device();
        const ScalarType type = x.scalar_type();
        if (code_of(type) < 0)
            value_error(std::string("x has dtype ") + c10::toString(type) +
                        ", expected bfloat16, float16 or float32");
        const int64_t rows = x.size(0), hidden = x.size(1);
        const bool quantize = a[4] == Py_True, keep = a[5] == Py_True;
        need(x, "x", type, {rows, hidden}, dev, true);
        const Tensor &w = need(a[1], "weight", type, {hidden}, dev);
        Tensor res, res_out, y, q, scales;
        if (a[3] != Py_None) {
            res = need(a[3], "residual", type, {rows, hidden}, dev, true);
            res_out = a[6] == Py_None ? fresh({rows, hidden}, type, dev)
                                      : need(a[6], "residual_out", type, {rows, hidden}, dev);
        } else if (a[6] != Py_None) {
            value_error("residual_out is given without residual");
        }
        if (!keep && !quantize) value_error("keep=False without quantize leaves no output");
        if (keep) y = fresh({rows, hidden}, type, dev);
        if (quantize) {
            q = fresh({rows, hidden}, kF8, dev);
            scales = fresh({rows, blocks(hidden)}, at::kFloat, dev);
        }
        if (rows)
            check(moeop_rms_norm(
                x.data_ptr(), row_stride(x), res.defined() ? res.data_ptr() : nullptr,
                res.defined() ? row_stride(res) : 0, w.data_ptr(), small(rows, "x"),
                small(hidden, "x"), code_of(type), (float)eps, keep ? y.data_ptr() : nullptr,
                res_out.defined() ? res_out.data_ptr() : nullptr,
                quantize ? ptr<uint8_t>(q) : nullptr, quantize ? ptr<float>(scales) : nullptr,
                stream_of(dev)));
        return Py_BuildValue("(NNNN)", wrapped(y), wrapped(res_out), wrapped(q), wrapped(scales));
    });
}

// (logits, top_k, scoring, bias, groups, group_limit, group_score, norm, factor)
PyObject *route_topk(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!counted(n, 9)) return nullptr;
    const long k = PyLong_AsLong(a[1]), scoring = PyLong_AsLong(a[2]), groups = PyLong_AsLong(a[4]),
               limit = PyLong_AsLong(a[5]), score = PyLong_AsLong(a[6]);
    const double factor = PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) return nullptr;
    return guarded([&] {
        const Tensor &x = first(a[0], "logits", 2);
        const at::Device dev = x.device();
        if (code_of(x.scalar_type()) < 0)
            value_error(std::string("logits has dtype ") + c10::toString(x.scalar_type()) +
                        ", expected float32, bfloat16 or float16");
        const int64_t rows = x.size(0), experts = x.size(1);
        need(x, "logits", x.scalar_type(), {rows, experts}, dev, true);
        const float *bias = nullptr;
        if (a[3] != Py_None) bias = ptr<float>(need(a[3], "bias", at::kFloat, {experts}, dev));
        if (k < 0) value_error("top_k=" + std::to_string(k) + " must not be negative");
        const Tensor ids = fresh({rows, k}, at::kInt, dev), wts = fresh({rows, k}, at::kFloat, dev);
        const moeop_route_config c{small(experts, "logits"), small(k, "top_k"), (int)scoring,
                                   small(groups, "groups"), small(limit, "group_limit"), (int)score,
                                   a[7] == Py_True, (float)factor, code_of(x.scalar_type())};
        check(moeop_route_topk(&c, x.data_ptr(), row_stride(x), bias, small(rows, "logits"),
                               ptr<int32_t>(ids), ptr<float>(wts), stream_of(dev)));
        return Py_BuildValue("(NN)", wrapped(ids), wrapped(wts));
    });
}

// (a, a_scales, b, b_scales, out_dtype code, out)
PyObject *matmul_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!counted(n, 6)) return nullptr;
    const long code = PyLong_AsLong(a[4]);
    if (PyErr_Occurred()) return nullptr;
    return guarded([&] {
        const Tensor &x = first(a[0], "a", 2), &w = first(a[2], "b", 2);
        const at::Device dev = x.device();
        const int64_t m = x.size(0), k = x.size(1), cols = w.size(0);
        need(x, "a", kF8, {m, k}, dev, true);
        need(w, "b", kF8, {cols, k}, dev, true);
        const Tensor &sa = need(a[1], "a_scales", at::kFloat, {m, blocks(k)}, dev);
        const Tensor &sb = need(a[3], "b_scales", at::kFloat, {blocks(cols), blocks(k)}, dev);
        const Tensor out = a[5] == Py_None
                               ? fresh({m, cols}, type_of(code), dev)
                               : need(a[5], "out", type_of(code), {m, cols}, dev);
        check(moeop_matmul_fp8(ptr<uint8_t>(x), row_stride(x), ptr<float>(sa), ptr<uint8_t>(w),
                               row_stride(w), ptr<float>(sb), small(m, "a"), small(cols, "b"),
                               small(k, "a"), out.data_ptr(), (int)code, stream_of(dev)));
        return wrapped(out);
    });
}

// (q, scales, ids, wts, gate, gate_scales, up, up_scales, down, down_scales, workspace, addend,
//  out)
PyObject *experts_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!counted(n, 13)) return nullptr;
    return guarded([&] {
        const Tensor &q = first(a[0], "q", 2), &gate = first(a[4], "gate", 3),
                     &ids = first(a[2], "ids", 2);
        const at::Device dev = q.device();
        const int64_t t = q.size(0), h = q.size(1), e = gate.size(0), i = gate.size(1),
                      k = ids.size(1);
        need(q, "q", kF8, {t, h}, dev);
        const Tensor &scales = need(a[1], "scales", at::kFloat, {t, blocks(h)}, dev);
        need(ids, "ids", at::kInt, {t, k}, dev);
        const Tensor &wts = need(a[3], "wts", at::kFloat, {t, k}, dev);
        need(gate, "gate", kF8, {e, i, h}, dev);
        const Tensor &gs = need(a[5], "gate_scales", at::kFloat, {e, blocks(i), blocks(h)}, dev);
        const Tensor &up = need(a[6], "up", kF8, {e, i, h}, dev);
        const Tensor &us = need(a[7], "up_scales", at::kFloat, {e, blocks(i), blocks(h)}, dev);
        const Tensor &down = need(a[8], "down", kF8, {e, h, i}, dev);
        const Tensor &ds = need(a[9], "down_scales", at::kFloat, {e, blocks(h), blocks(i)}, dev);
        const uint16_t *addend = nullptr;
        if (a[11] != Py_None)
            addend = ptr<uint16_t>(need(a[11], "addend", at::kBFloat16, {t, h}, dev));
        const Tensor out = a[12] == Py_None ? fresh({t, h}, at::kBFloat16, dev)
                                            : need(a[12], "out", at::kBFloat16, {t, h}, dev);
        const moeop_experts_config c{small(h, "q"), small(i, "gate"), small(e, "gate"),
                                     small(k, "ids")};
        Tensor ws;
        if (a[10] == Py_None) {
            const size_t bytes = moeop_experts_workspace_size(&c, small(t, "q"));
            if (!bytes) throw Status{MOE_ERR_INVALID_ARG};
            ws = fresh({(int64_t)bytes}, at::kByte, dev);
        } else {
            ws = tensor(a[10], "the workspace");
            if (ws.device() != dev)
                value_error("the workspace is on " + ws.device().str() + ", expected " + dev.str());
        }
        const moeop_experts_weights w{ptr<uint8_t>(gate), ptr<uint8_t>(up), ptr<uint8_t>(down),
                                      ptr<float>(gs), ptr<float>(us), ptr<float>(ds)};
        check(moeop_experts_fp8(&c, &w, ptr<uint8_t>(q), ptr<float>(scales), ptr<int32_t>(ids),
                                ptr<float>(wts), addend, ptr<uint16_t>(out), small(t, "q"),
                                ws.data_ptr(), (size_t)ws.numel(), stream_of(dev)));
        return wrapped(out);
    });
}

PyObject *set_error_class(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XDECREF(g_moe_error);
    g_moe_error = cls;
    Py_RETURN_NONE;
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(rms_norm), FAST(route_topk), FAST(matmul_fp8), FAST(experts_fp8),
                           {"set_error_class", set_error_class, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_moe_ops", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_ops(void) { return PyModule_Create(&g_module); }
