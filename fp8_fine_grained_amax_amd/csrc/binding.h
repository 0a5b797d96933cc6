// What the Python bindings share: checks of tensors, allocation of outputs, errors. The entry points that other files
// define for the module's table are declared at the end.
#pragma once
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/record_function.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <string>
#include <vector>

#include "fp8fg.h"

inline PyObject* g_error = nullptr;      // the package's exception type
inline thread_local bool g_watched = false;      // watched() at the entry of this thread's call: once, as it takes 0.05 us

// A Python exception is set; unwinds to the entry. One type for all files: the entries are in another file than some of the
// functions that throw it.
struct Raised {};

namespace {

[[noreturn]] void fail(const char* format, ...) {
    char text[600];
    va_list args;
    va_start(args, format);
    vsnprintf(text, sizeof text, format, args);
    va_end(args);
    PyErr_SetString(g_error, text);
    throw Raised{};
}

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kByte: return "uint8";
        case at::kInt: return "int32";
        case at::kLong: return "int64";
        case at::kFloat: return "float32";
        case at::kDouble: return "float64";
        case at::kHalf: return "float16";
        case at::kBFloat16: return "bfloat16";
        default: return c10::toString(t);
    }
}

std::string shape_text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); i++) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

bool is_none(PyObject* o) { return o == Py_None; }

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) fail("%s must be a torch tensor", what);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) fail("fp8fg operates on GPU tensors only (%s)", what);
    return t;
}

const at::Tensor& dims(PyObject* o, const char* what, int64_t n) {
    const at::Tensor& t = tensor(o, what);
    if (t.dim() != n) fail("%s must have %d dimensions, got %d", what, (int)n, (int)t.dim());
    return t;
}

void same_device(const at::Tensor& t, const char* what, c10::Device d) {
    if (t.device() != d) fail("%s is on cuda:%d, the first argument on cuda:%d", what, (int)t.device().index(), (int)d.index());
}

// A contiguous tensor of this type and shape.
void* dense(const at::Tensor& t, const char* what, at::ScalarType type, at::IntArrayRef shape, c10::Device d) {
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
        fail("%s must be a contiguous %s tensor of shape %s, got %s %s with strides %s", what, type_name(type),
             shape_text(shape).c_str(), type_name(t.scalar_type()), shape_text(t.sizes()).c_str(), shape_text(t.strides()).c_str());
    same_device(t, what, d);
    return t.data_ptr();
}
void* dense(PyObject* o, const char* what, at::ScalarType type, at::IntArrayRef shape, c10::Device d) {
    return dense(tensor(o, what), what, type, shape, d);
}

int real_type(const at::Tensor& t, const char* what) {
    if (t.scalar_type() == at::kFloat) return FG_OUT_F32;
    if (t.scalar_type() == at::kBFloat16) return FG_OUT_BF16;
    fail("%s must be float32 or bfloat16, got %s", what, type_name(t.scalar_type()));
}

// Row stride of a row-major matrix whose rows may be further apart than they are wide.
int64_t matrix(const at::Tensor& t, const char* what, int64_t rows, int64_t cols, c10::Device d) {
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        fail("%s must have shape (%lld, %lld), got %s", what, (long long)rows, (long long)cols, shape_text(t.sizes()).c_str());
    same_device(t, what, d);
    if (rows == 0 || cols == 0) return cols;                  // nothing is read, whatever the strides
    if ((cols > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < cols))
        fail("%s must have unit column stride and rows that do not overlap, got strides %s", what, shape_text(t.strides()).c_str());
    return rows > 1 ? t.stride(0) : cols;                     // a single row has no stride between rows
}

int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
int flag(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v;
}
fg_scale_mode mode(PyObject* pow2) { return flag(pow2) ? FG_SCALE_POW2 : FG_SCALE_FP32; }

// Whether somebody is to see an allocation: a dispatch mode or another layer of this thread, a profiler, or torch's fill of new
// memory in its deterministic mode.
bool watched() {
    return !(c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set).empty() || at::hasCallbacks() ||
           at::globalContext().deterministicAlgorithms();
}
// Held over a call, whose allocations may themselves call Python, and that another call.
struct Watch {
    const bool before = g_watched;
    Watch() { g_watched = watched(); }
    ~Watch() { g_watched = before; }
};
// Past torch's dispatcher where nobody watches, as it took 0.2 of 0.65 us a tensor.
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, c10::Device d) {
    if (g_watched) return at::empty(shape, at::TensorOptions(type).device(d));
    return at::Tensor(at::detail::empty_cuda(shape, type, d, std::nullopt));
}
// The caller's output buffer, or a new one.
at::Tensor output(PyObject* o, const char* what, at::ScalarType type, at::IntArrayRef shape, c10::Device d) {
    if (is_none(o)) return make(shape, type, d);
    const at::Tensor& t = tensor(o, what);
    dense(t, what, type, shape, d);
    return t;
}

at::Tensor workspace(PyObject* o, int64_t need, c10::Device d) {
    if (is_none(o)) return make({need}, at::kByte, d);
    const at::Tensor& t = tensor(o, "workspace");
    if (t.scalar_type() != at::kByte || !t.is_contiguous()) fail("workspace must be a contiguous uint8 tensor");
    same_device(t, "workspace", d);
    return t;
}

hipStream_t stream(c10::Device d) { return c10::hip::getCurrentHIPStream(d.index()).stream(); }

void check(fg_status s, const char* what) {
    if (s == FG_OK) return;
    if (s == FG_ERR_HIP) fail("%s: %s (hipError %d)", what, fg_status_string(s), fg_last_hip_error());
    fail("%s: %s", what, fg_status_string(s));
}

// A library call with the interpreter's lock released: a launch waits where the queue is full.
template <class Call>
void run(const char* what, Call&& call) {
    PyThreadState* state = PyEval_SaveThread();
    const fg_status s = call();
    PyEval_RestoreThread(state);
    check(s, what);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

PyObject* tuple(const std::vector<at::Tensor>& v) {
    PyObject* r = PyTuple_New((Py_ssize_t)v.size());
    if (!r) throw Raised{};
    for (size_t i = 0; i < v.size(); i++) {
        PyObject* o = v[i].defined() ? THPVariable_Wrap(v[i]) : (Py_INCREF(Py_None), Py_None);
        if (!o) {
            Py_DECREF(r);
            throw Raised{};
        }
        PyTuple_SET_ITEM(r, (Py_ssize_t)i, o);
    }
    return r;
}

}  // namespace

// In train_binding.cpp; they throw as the helpers above do.
PyObject* fg_py_norm_quantize(PyObject* const* a);
PyObject* fg_py_norm_bwd(PyObject* const* a);
PyObject* fg_py_orthogonalize(PyObject* const* a);
