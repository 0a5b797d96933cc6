// Python binding of the feed-forward operators (module _ffn, called by ffn.py): the same job as the ctypes binding of
// the other entry points (checks of the tensors, allocation of what the caller does not pass, torch's current stream
// of the tensors' own device) in compiled code, because at a few tokens the interpreter takes longer over it than the
// kernels take: a call with its outputs cost 10 us (the Linear, one output) to 27 us (the activation's backward, seven)
// in Python, against 4 to 11 us of kernels; here 5 and 16.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <string>
#include <vector>

#include "fp8fg_ffn.h"

namespace {

PyObject* g_error = nullptr;      // the package's exception type

// A Python exception is set; unwinds to the entry.
struct Raised {};

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
fg_act activation(PyObject* o) {
    const int64_t a = whole(o);
    if (a < FG_ACT_NONE || a > FG_ACT_SILU) fail("unknown activation %lld", (long long)a);
    return (fg_act)a;
}
fg_scale_mode mode(PyObject* pow2) { return flag(pow2) ? FG_SCALE_POW2 : FG_SCALE_FP32; }

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, c10::Device d) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(d));
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

// xq, sx, wq, sw, bias, act, residual, out_bf16, y, pow2
PyObject* linear(PyObject* const* a) {
    const at::Tensor &xq = dims(a[0], "xq", 2), &wq = dims(a[2], "wq", 2);
    const c10::Device d = xq.device();
    const int64_t M = xq.size(0), K = xq.size(1), N = wq.size(0);
    const auto* x = (const uint8_t*)dense(xq, "xq", at::kByte, {M, K}, d);
    const auto* w = (const uint8_t*)dense(wq, "wq", at::kByte, {N, K}, d);
    const at::Tensor &sx = tensor(a[1], "sx"), &sw = tensor(a[3], "sw");
    if (K % 128 == 0) {                                       // the library refuses others
        dense(sx, "sx", at::kFloat, {K / 128, M}, d);
        dense(sw, "sw", at::kFloat, {cdiv(N, 128), K / 128}, d);
    }
    const void *bias = nullptr, *residual = nullptr;
    int bias_type = 0, res_type = 0;
    int64_t ld_res = N;
    if (!is_none(a[4])) {
        const at::Tensor& b = tensor(a[4], "bias");
        bias_type = real_type(b, "bias");
        bias = dense(b, "bias", b.scalar_type(), {N}, d);
    }
    if (!is_none(a[6])) {
        const at::Tensor& r = tensor(a[6], "residual");
        res_type = real_type(r, "residual");
        ld_res = matrix(r, "residual", M, N, d);
        residual = r.data_ptr();
    }
    const fg_act act = activation(a[5]);
    at::ScalarType type = flag(a[7]) ? at::kBFloat16 : at::kFloat;
    if (!is_none(a[8])) {
        real_type(tensor(a[8], "y"), "y");
        type = tensor(a[8], "y").scalar_type();
    }
    const c10::DeviceGuard guard(d);
    const at::Tensor y = output(a[8], "y", type, {M, N}, d);
    const fg_scale_mode scales = mode(a[9]);
    const hipStream_t on = stream(d);
    run("fg_fp8_gemm_fprop_epilogue", [&] {
        return fg_fp8_gemm_fprop_epilogue(x, (const float*)sx.data_ptr(), w, (const float*)sw.data_ptr(), M, N, K, bias,
                                          (fg_out_dtype)bias_type, act, residual, (fg_out_dtype)res_type, ld_res, y.data_ptr(),
                                          type == at::kBFloat16 ? FG_OUT_BF16 : FG_OUT_F32, scales, on);
    });
    return THPVariable_Wrap(y);
}

// z, act, gated, pow2, zq, sz, aq, sa
PyObject* act_forward(PyObject* const* a) {
    const at::Tensor& z = dims(a[0], "z", 2);
    const c10::Device d = z.device();
    const int64_t rows = z.size(0), W = z.size(1);
    const int gated = flag(a[2]);
    if (gated && W % 2) fail("a gated z has an even width, got %lld", (long long)W);
    if (z.scalar_type() != at::kBFloat16) fail("z must be bfloat16, got %s", type_name(z.scalar_type()));
    const int64_t F = gated ? W / 2 : W, ld = matrix(z, "z", rows, W, d);
    const fg_act act = activation(a[1]);
    const c10::DeviceGuard guard(d);
    const at::Tensor zq = output(a[4], "zq", at::kByte, {rows, W}, d);
    const at::Tensor sz = output(a[5], "sz", at::kFloat, {cdiv(W, 128), rows}, d);
    const at::Tensor aq = output(a[6], "aq", at::kByte, {rows, F}, d);
    const at::Tensor sa = output(a[7], "sa", at::kFloat, {cdiv(F, 128), rows}, d);
    const fg_scale_mode scales = mode(a[3]);
    const hipStream_t on = stream(d);
    run("fg_act_checkpoint_fwd", [&] {
        return fg_act_checkpoint_fwd(z.data_ptr(), rows, F, ld, act, gated, scales, (uint8_t*)zq.data_ptr(), (float*)sz.data_ptr(),
                                     (uint8_t*)aq.data_ptr(), (float*)sa.data_ptr(), on);
    });
    return tuple({zq, sz, aq, sa});
}

// zq, sz, da, act, gated, pow2, token_tiles, recompute, bias_grad, out (7 or None), workspace
PyObject* act_backward(PyObject* const* a) {
    const at::Tensor& zq = dims(a[0], "zq", 2);
    const c10::Device d = zq.device();
    const int64_t rows = zq.size(0), W = zq.size(1);
    const int gated = flag(a[4]);
    if (gated && W % 2) fail("a gated checkpoint has an even width, got %lld", (long long)W);
    const int64_t F = gated ? W / 2 : W;
    dense(zq, "zq", at::kByte, {rows, W}, d);
    const auto* sz = (const float*)dense(a[1], "sz", at::kFloat, {cdiv(W, 128), rows}, d);
    const at::Tensor& da = tensor(a[2], "da");
    const int da_type = real_type(da, "da");
    const int64_t ld = matrix(da, "da", rows, F, d);
    const fg_act act = activation(a[3]);
    PyObject* given[7] = {Py_None, Py_None, Py_None, Py_None, Py_None, Py_None, Py_None};
    if (!is_none(a[9])) {
        if (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != 7) fail("out must be an ActGrad");
        for (int i = 0; i < 7; i++) given[i] = PyTuple_GET_ITEM(a[9], i);
    }
    const c10::DeviceGuard guard(d);
    const int64_t tiles = cdiv(rows, 128);
    at::Tensor qr, sr, ar, sa, db, ws;
    const at::Tensor qc = output(given[0], "dzq_cols", at::kByte, {rows, W}, d);
    const at::Tensor sc = output(given[1], "sdz_cols", at::kFloat, {cdiv(W, 128), rows}, d);
    if (flag(a[6])) {
        qr = output(given[2], "dzq_rows", at::kByte, {W, rows}, d);
        sr = output(given[3], "sdz_rows", at::kFloat, {tiles, W}, d);
    }
    if (flag(a[7])) {
        ar = output(given[4], "aq_rows", at::kByte, {F, rows}, d);
        sa = output(given[5], "sa_rows", at::kFloat, {tiles, F}, d);
    }
    int64_t need = 0;
    if (flag(a[8])) {
        db = output(given[6], "dbias", at::kFloat, {W}, d);
        need = fg_act_checkpoint_bwd_workspace(rows, F, gated);
    }
    if (need || !is_none(a[10])) ws = workspace(a[10], need, d);
    auto at_ = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    const fg_scale_mode scales = mode(a[5]);
    const hipStream_t on = stream(d);
    run("fg_act_checkpoint_bwd", [&] {
        return fg_act_checkpoint_bwd((const uint8_t*)zq.data_ptr(), sz, da.data_ptr(), (fg_out_dtype)da_type, ld, rows, F, act, gated,
                                     scales, (uint8_t*)qc.data_ptr(), (float*)sc.data_ptr(), (uint8_t*)at_(qr), (float*)at_(sr),
                                     (uint8_t*)at_(ar), (float*)at_(sa), (float*)at_(db), at_(ws), ws.defined() ? ws.numel() : 0, on);
    });
    return tuple({qc, sc, qr, sr, ar, sa, db});
}

// x, ids, weights, w1q, s1, w2q, s2, act, out_bf16, y, pow2, workspace
PyObject* moe(PyObject* const* a) {
    const at::Tensor &x = dims(a[0], "x", 2), &ids = dims(a[1], "ids", 2), &w1 = dims(a[3], "w1q", 3);
    const c10::Device d = x.device();
    const int64_t T = x.size(0), H = x.size(1), topk = ids.size(1), E = w1.size(0), I2 = w1.size(1), I = I2 / 2;
    if (I2 % 2) fail("w1q holds gate and up rows: an even number of them, got %lld", (long long)I2);
    if (topk > INT32_MAX || E > INT32_MAX) fail("ids and w1q have more columns or experts than 32 bits count");
    if (x.scalar_type() != at::kBFloat16) fail("x must be bfloat16, got %s", type_name(x.scalar_type()));
    const int64_t ld_x = matrix(x, "x", T, H, d);
    const auto* id = (const int32_t*)dense(ids, "ids", at::kInt, {T, topk}, d);
    const auto* weights = (const float*)dense(a[2], "weights", at::kFloat, {T, topk}, d);
    const auto* w1q = (const uint8_t*)dense(w1, "w1q", at::kByte, {E, I2, H}, d);
    const auto* w2q = (const uint8_t*)dense(a[5], "w2q", at::kByte, {E, H, I}, d);
    const at::Tensor &s1 = tensor(a[4], "s1"), &s2 = tensor(a[6], "s2");
    if (H % 128 == 0 && I % 128 == 0) {                       // the library refuses others
        dense(s1, "s1", at::kFloat, {E, I2 / 128, H / 128}, d);
        dense(s2, "s2", at::kFloat, {E, H / 128, I / 128}, d);
    }
    const fg_act act = activation(a[7]);
    const c10::DeviceGuard guard(d);
    const at::Tensor y = is_none(a[9]) ? make({T, H}, flag(a[8]) ? at::kBFloat16 : at::kFloat, d) : tensor(a[9], "y");
    const int out = real_type(y, "y");
    const int64_t ld_y = matrix(y, "y", T, H, d);
    const at::Tensor ws = workspace(a[11], fg_moe_few_tokens_workspace(T, (int32_t)topk, H, I), d);
    const fg_scale_mode scales = mode(a[10]);
    const hipStream_t on = stream(d);
    run("fg_moe_few_tokens", [&] {
        return fg_moe_few_tokens(x.data_ptr(), ld_x, id, weights, T, (int32_t)topk, w1q, (const float*)s1.data_ptr(), w2q,
                                 (const float*)s2.data_ptr(), (int32_t)E, H, I, act, scales, ws.data_ptr(), ws.numel(), y.data_ptr(),
                                 ld_y, (fg_out_dtype)out, on);
    });
    return THPVariable_Wrap(y);
}

// Entry: the number of arguments, and C++ errors as Python's.
template <PyObject* (*F)(PyObject* const*), int ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != ARGS) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", ARGS, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised&) {
    } catch (const c10::OutOfMemoryError& e) {                // torch's own, for callers that free and try again
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XDECREF(g_error);
    g_error = type;
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int ARGS>
constexpr PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void*)(PyObject * (*)(PyObject*, PyObject* const*, Py_ssize_t)) entry<F, ARGS>, METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<linear, 10>("linear"),
    method<act_forward, 8>("act_forward"),
    method<act_backward, 11>("act_backward"),
    method<moe, 12>("moe"),
    {"set_error", set_error, METH_O, "The exception type that failed checks raise."},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ffn", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ffn() {
    g_error = PyExc_RuntimeError;
    Py_INCREF(g_error);
    return PyModule_Create(&g_module);
}
