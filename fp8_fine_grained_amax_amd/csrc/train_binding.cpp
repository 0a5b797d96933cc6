// Python binding of the operators at the two ends of a Linear's training step (module _ffn, called by train.py): as in
// ffn_binding.cpp, in compiled code because small calls' kernels take less time than an interpreted binding.
#include "binding.h"
#include "fp8fg_train.h"

namespace {

double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

fg_norm_kind norm_kind(PyObject* o) {
    const int64_t k = whole(o);
    if (k != FG_NORM_LAYER && k != FG_NORM_RMS) fail("unknown norm %lld", (long long)k);
    return (fg_norm_kind)k;
}

void* data(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

}  // namespace

// x, gamma, beta, kind, eps, pow2, token_tiles, with_y, statistics, q_cols, s_cols, q_rows, s_rows, y, mean, rstd
PyObject* fg_py_norm_quantize(PyObject* const* a) {
    const at::Tensor& x = dims(a[0], "x", 2);
    const c10::Device d = x.device();
    const int64_t rows = x.size(0), cols = x.size(1);
    const int x_type = real_type(x, "x");
    const int64_t ld = matrix(x, "x", rows, cols, d);
    const at::Tensor& g = tensor(a[1], "gamma");
    const int w_type = real_type(g, "gamma");
    const void* gamma = dense(g, "gamma", g.scalar_type(), {cols}, d);
    const void* beta = is_none(a[2]) ? nullptr : dense(a[2], "beta", g.scalar_type(), {cols}, d);
    const fg_norm_kind kind = norm_kind(a[3]);
    const float eps = (float)real(a[4]);
    const fg_scale_mode scales = mode(a[5]);
    const int tokens = flag(a[6]), with_y = flag(a[7]), statistics = flag(a[8]) || tokens;
    const c10::DeviceGuard guard(d);
    at::Tensor qr, sr, y, mean, rstd;
    const at::Tensor qc = output(a[9], "q_cols", at::kByte, {rows, cols}, d);
    const at::Tensor sc = output(a[10], "s_cols", at::kFloat, {cdiv(cols, 128), rows}, d);
    if (tokens) {
        qr = output(a[11], "q_rows", at::kByte, {cols, rows}, d);
        sr = output(a[12], "s_rows", at::kFloat, {cdiv(rows, 128), cols}, d);
    }
    if (with_y) y = output(a[13], "y", at::kBFloat16, {rows, cols}, d);
    if (statistics) {
        if (kind == FG_NORM_LAYER) mean = output(a[14], "mean", at::kFloat, {rows}, d);
        rstd = output(a[15], "rstd", at::kFloat, {rows}, d);
    }
    const hipStream_t on = stream(d);
    run("fg_norm_quantize", [&] {
        return fg_norm_quantize(x.data_ptr(), (fg_out_dtype)x_type, ld, rows, cols, kind, gamma, beta, (fg_out_dtype)w_type, eps, scales,
                                (uint8_t*)qc.data_ptr(), (float*)sc.data_ptr(), (uint8_t*)data(qr), (float*)data(sr), data(y),
                                (float*)data(mean), (float*)data(rstd), on);
    });
    return tuple({qc, sc, qr, sr, y, mean, rstd});
}

// x, mean, rstd, gamma, dy, residual_grad, kind, dx_bf16, weight_grad, bias_grad, accumulate, dx, out (dgamma, dbeta), workspace
PyObject* fg_py_norm_bwd(PyObject* const* a) {
    const at::Tensor& x = dims(a[0], "x", 2);
    const c10::Device d = x.device();
    const int64_t rows = x.size(0), cols = x.size(1);
    const int x_type = real_type(x, "x");
    const int64_t ld_x = matrix(x, "x", rows, cols, d);
    const fg_norm_kind kind = norm_kind(a[6]);
    const float* mean = nullptr;
    if (kind == FG_NORM_LAYER) mean = (const float*)dense(a[1], "mean", at::kFloat, {rows}, d);
    const auto* rstd = (const float*)dense(a[2], "rstd", at::kFloat, {rows}, d);
    const at::Tensor& g = tensor(a[3], "gamma");
    const int w_type = real_type(g, "gamma");
    const void* gamma = dense(g, "gamma", g.scalar_type(), {cols}, d);
    const at::Tensor& dy = tensor(a[4], "dy");
    const int dy_type = real_type(dy, "dy");
    const int64_t ld_dy = matrix(dy, "dy", rows, cols, d);
    const void* dres = nullptr;
    int dres_type = 0;
    int64_t ld_dres = cols;
    if (!is_none(a[5])) {
        const at::Tensor& r = tensor(a[5], "residual_grad");
        dres_type = real_type(r, "residual_grad");
        ld_dres = matrix(r, "residual_grad", rows, cols, d);
        dres = r.data_ptr();
    }
    at::ScalarType type = flag(a[7]) ? at::kBFloat16 : at::kFloat;
    if (!is_none(a[11])) {
        real_type(tensor(a[11], "dx"), "dx");
        type = tensor(a[11], "dx").scalar_type();
    }
    const int weight = flag(a[8]), bias = flag(a[9]), accumulate = flag(a[10]);
    PyObject* given[2] = {Py_None, Py_None};
    if (!is_none(a[12])) {
        if (!PyTuple_Check(a[12]) || PyTuple_GET_SIZE(a[12]) != 2) fail("out must be a pair");
        for (int i = 0; i < 2; i++) given[i] = PyTuple_GET_ITEM(a[12], i);
    }
    if (accumulate && ((weight && is_none(given[0])) || (bias && is_none(given[1])))) fail("accumulate needs existing gradients");
    const c10::DeviceGuard guard(d);
    const at::Tensor dx = output(a[11], "dx", type, {rows, cols}, d);
    at::Tensor dgamma, dbeta, ws;
    if (weight) dgamma = output(given[0], "dgamma", at::kFloat, {cols}, d);
    if (bias) dbeta = output(given[1], "dbeta", at::kFloat, {cols}, d);
    const int64_t need = weight || bias ? fg_norm_bwd_workspace(rows, cols) : 0;
    if (need || !is_none(a[13])) ws = workspace(a[13], need, d);
    const hipStream_t on = stream(d);
    run("fg_norm_bwd", [&] {
        return fg_norm_bwd(x.data_ptr(), (fg_out_dtype)x_type, ld_x, mean, rstd, gamma, (fg_out_dtype)w_type, dy.data_ptr(),
                           (fg_out_dtype)dy_type, ld_dy, dres, (fg_out_dtype)dres_type, ld_dres, rows, cols, kind, dx.data_ptr(),
                           type == at::kBFloat16 ? FG_OUT_BF16 : FG_OUT_F32, (float*)data(dgamma), (float*)data(dbeta), accumulate,
                           data(ws), ws.defined() ? ws.numel() : 0, on);
    });
    return tuple({dx, dgamma, dbeta});
}

// g, steps, a, b, c, eps, scale, out, workspace
PyObject* fg_py_orthogonalize(PyObject* const* a) {
    const at::Tensor& g = tensor(a[0], "g");
    const c10::Device d = g.device();
    if (g.dim() != 2 && g.dim() != 3) fail("g must have 2 or 3 dimensions, got %d", (int)g.dim());
    const int type = real_type(g, "g");
    const int64_t batch = g.dim() == 3 ? g.size(0) : 1, N = g.size(-2), K = g.size(-1);
    int64_t ld = K;
    if (g.numel() > 0) {
        if (N > 1) ld = g.stride(-2);
        else if (batch > 1) ld = g.stride(0);                 // matrices of one row: the matrices' distance
        if ((K > 1 && g.stride(-1) != 1) || ld < K || (batch > 1 && g.stride(0) != N * ld))
            fail("g must have unit column stride, rows that do not overlap and matrices one behind the other, got strides %s",
                 shape_text(g.strides()).c_str());
    }
    const int64_t steps = whole(a[1]);
    if (steps < 1 || steps > INT32_MAX) fail("steps must be a positive number, got %lld", (long long)steps);
    const float fa = (float)real(a[2]), fb = (float)real(a[3]), fc = (float)real(a[4]), eps = (float)real(a[5]), scale = (float)real(a[6]);
    const c10::DeviceGuard guard(d);
    const at::Tensor out = output(a[7], "out", at::kBFloat16, g.sizes(), d);
    const at::Tensor ws = workspace(a[8], fg_orthogonalize_workspace(batch, N, K), d);
    const hipStream_t on = stream(d);
    run("fg_orthogonalize", [&] {
        return fg_orthogonalize(g.data_ptr(), (fg_out_dtype)type, ld, batch, N, K, (int)steps, fa, fb, fc, eps, scale, out.data_ptr(),
                                ws.data_ptr(), ws.numel(), on);
    });
    return THPVariable_Wrap(out);
}
