// Python binding of the feed-forward operators (module _ffn, called by ffn.py): the same job as the ctypes binding of
// the other entry points (checks of the tensors, allocation of what the caller does not pass, torch's current stream
// of the tensors' own device) in compiled code, because at a few tokens the interpreter takes longer over it than the
// kernels take: a call with its outputs cost 10 us (the Linear, one output) to 27 us (the activation's backward, seven)
// in Python, against 4 to 11 us of kernels; here 5 and 13.
#include "binding.h"
#include "fp8fg_ffn.h"

namespace {

fg_act activation(PyObject* o) {
    const int64_t a = whole(o);
    if (a < FG_ACT_NONE || a > FG_ACT_SILU) fail("unknown activation %lld", (long long)a);
    return (fg_act)a;
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
    const Watch watch;
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
    method<fg_py_norm_quantize, 16>("norm_quantize"),
    method<fg_py_norm_bwd, 14>("norm_bwd"),
    method<fg_py_orthogonalize, 9>("orthogonalize"),
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
