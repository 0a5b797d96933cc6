"""Binding of the feed-forward operators (include/fp8fg_ffn.h): the functions carry the C names, check their
tensors, allocate outputs and workspaces the caller does not pass, and run on torch's current stream of the
tensors' own device, whichever device is current."""
import ctypes
from typing import NamedTuple, Optional

import torch

from . import Fp8fgError, _check, _mode, _out_code, lib

FG_ACT_NONE, FG_ACT_RELU, FG_ACT_GELU_TANH, FG_ACT_SILU = 0, 1, 2, 3


def declare(L):
    """Argument types of the feed-forward entry points."""
    P, I64, I, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int32
    L.fg_fp8_gemm_fprop_epilogue.argtypes = [P, P, P, P, I64, I64, I64, P, I, I, P, I, I64, P, I, I, P]
    L.fg_act_checkpoint_fwd.argtypes = [P, I64, I64, I64, I, I, I, P, P, P, P, P]
    L.fg_act_checkpoint_bwd.argtypes = [P, P, P, I, I64, I64, I64, I, I, I, P, P, P, P, P, P, P, P, I64, P]
    L.fg_moe_few_tokens.argtypes = [P, I64, P, P, I64, I32, P, P, P, P, I32, I64, I64, I, I, P, I64, P, I64, I, P]
    for f in ("fg_fp8_gemm_fprop_epilogue", "fg_act_checkpoint_fwd", "fg_act_checkpoint_bwd", "fg_moe_few_tokens"):
        getattr(L, f).restype = I
    L.fg_act_checkpoint_bwd_workspace.argtypes = [I64, I64, I]
    L.fg_moe_few_tokens_workspace.argtypes = [I64, I32, I64, I64]
    for f in ("fg_act_checkpoint_bwd_workspace", "fg_moe_few_tokens_workspace"):
        getattr(L, f).restype = I64


def _fail(text):
    raise Fp8fgError(text)


def _name(dtype):
    return str(dtype).replace("torch.", "")


def _device(x):
    """Index of the GPU that holds x: the call runs there, on torch's current stream of it."""
    d = x.get_device()
    if d < 0:
        _fail("fp8fg operates on GPU tensors only")
    return d


def _dense(t, what, dtype, shape, dev):
    """A contiguous tensor of this type and shape on GPU `dev`."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _fail(f"{what} must be a contiguous {_name(dtype)} tensor of shape {tuple(shape)}, got {_name(t.dtype)} "
              f"{tuple(t.shape)} with strides {t.stride()}")
    if t.get_device() != dev:
        _fail(f"{what} is on {t.device}, the first argument on cuda:{dev}")
    return t


_REAL = (torch.float32, torch.bfloat16)


def _matrix(t, what, dtypes, shape, dev):
    """Row stride of a row-major matrix whose rows may be further apart than they are wide."""
    if t.dtype not in dtypes or t.shape != shape:
        _fail(f"{what} must be a {' or '.join(map(_name, dtypes))} matrix of shape {tuple(shape)}, got {_name(t.dtype)} "
              f"{tuple(t.shape)}")
    if t.get_device() != dev:
        _fail(f"{what} is on {t.device}, the first argument on cuda:{dev}")
    rows, cols = shape
    ld, step = t.stride()
    if rows == 0 or cols == 0:
        return cols                                  # nothing is read, whatever the strides
    if (cols > 1 and step != 1) or (rows > 1 and ld < cols):
        _fail(f"{what} must have unit column stride and rows that do not overlap, got strides {t.stride()}")
    return ld if rows > 1 else cols                  # a single row has no stride between rows


def _out(t, what, dtype, shape, like, dev):
    return torch.empty(shape, dtype=dtype, device=like.device) if t is None else _dense(t, what, dtype, shape, dev)


def _act_code(act):
    if act not in (FG_ACT_NONE, FG_ACT_RELU, FG_ACT_GELU_TANH, FG_ACT_SILU):
        _fail(f"unknown activation {act!r}")
    return int(act)


def _dims(t, what, n):
    if t.dim() != n:
        _fail(f"{what} must have {n} dimensions, got {t.dim()}")
    return t.shape


def _workspace(t, need, like, dev):
    if t is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    if t.dtype is not torch.uint8 or not t.is_contiguous() or t.get_device() != dev:
        _fail(f"workspace must be a contiguous uint8 tensor on cuda:{dev}")
    return t


def _addr(t):
    return None if t is None else t.data_ptr()


def _run(function, dev, *args):
    """One library call on GPU `dev` and torch's current stream there. The raw stream handle and the device's index are
    what torch's own launchers use; their public wrappers cost as much as a kernel of few tokens."""
    f = getattr(lib(), function)
    if torch._C._cuda_getDevice() == dev:
        status = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status != 0:
        _check(status, function)


def _cdiv(a, b):
    return (a + b - 1) // b


def fg_fp8_gemm_fprop_epilogue(xq, sx, wq, sw, bias=None, act: int = FG_ACT_NONE, residual=None, out_dtype=torch.bfloat16,
                               y=None, pow2: bool = False):
    """Y [M, N] = act(X [M, K] . W [N, K]^T + bias [N]) + residual [M, N] from E4M3 codes and their scales. bias and
    residual: float32 or bfloat16; residual may have a row stride, and may be y itself."""
    dev = _device(xq)
    M, K = _dims(xq, "xq", 2)
    N = _dims(wq, "wq", 2)[0]
    _dense(xq, "xq", torch.uint8, (M, K), dev)
    _dense(wq, "wq", torch.uint8, (N, K), dev)
    if K % 128 == 0:                                 # the library refuses others
        _dense(sx, "sx", torch.float32, (K // 128, M), dev)
        _dense(sw, "sw", torch.float32, (_cdiv(N, 128), K // 128), dev)
    bias_type = res_type = 0
    if bias is not None:
        bias_type = _out_code(_dense(bias, "bias", bias.dtype, (N,), dev).dtype)
    ld_res = N
    if residual is not None:
        ld_res = _matrix(residual, "residual", _REAL, (M, N), dev)
        res_type = _out_code(residual.dtype)
    y = _out(y, "y", out_dtype if y is None else y.dtype, (M, N), xq, dev)
    _run("fg_fp8_gemm_fprop_epilogue", dev, xq.data_ptr(), _addr(sx), wq.data_ptr(), _addr(sw), M, N, K, _addr(bias),
         bias_type, _act_code(act), _addr(residual), res_type, ld_res, y.data_ptr(), _out_code(y.dtype), _mode(pow2))
    return y


def fg_act_checkpoint_fwd(z, act: int, gated: bool = False, pow2: bool = False, zq=None, sz=None, aq=None, sa=None):
    """a = act(z), or act(gate) * up with z = [gate | up], from bf16 z [rows, W]: returns (zq u8 [rows, W], sz f32
    [W/128, rows], aq u8 [rows, F], sa f32 [F/128, rows]), the checkpoint of z and a, both in 1x128 tiles along the
    columns. F = W / 2 when gated, else W."""
    dev = _device(z)
    rows, W = _dims(z, "z", 2)
    if gated and W % 2:
        _fail(f"a gated z has an even width, got {W}")
    F = W // 2 if gated else W
    ld = _matrix(z, "z", (torch.bfloat16,), (rows, W), dev)
    zq = _out(zq, "zq", torch.uint8, (rows, W), z, dev)
    sz = _out(sz, "sz", torch.float32, (_cdiv(W, 128), rows), z, dev)
    aq = _out(aq, "aq", torch.uint8, (rows, F), z, dev)
    sa = _out(sa, "sa", torch.float32, (_cdiv(F, 128), rows), z, dev)
    _run("fg_act_checkpoint_fwd", dev, z.data_ptr(), rows, F, ld, _act_code(act), int(bool(gated)), _mode(pow2),
         zq.data_ptr(), sz.data_ptr(), aq.data_ptr(), sa.data_ptr())
    return zq, sz, aq, sa


class ActGrad(NamedTuple):
    """What fg_act_checkpoint_bwd returns: dz [rows, W] in both tilings, a [rows, F] in tiles along the rows, and the
    column sums of dz; None for what was not asked for."""
    dzq_cols: torch.Tensor
    sdz_cols: torch.Tensor
    dzq_rows: Optional[torch.Tensor]
    sdz_rows: Optional[torch.Tensor]
    aq_rows: Optional[torch.Tensor]
    sa_rows: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


def fg_act_checkpoint_bwd(zq, sz, da, act: int, gated: bool = False, pow2: bool = False, token_tiles: bool = True,
                          recompute: bool = True, bias_grad: bool = False, out: Optional[ActGrad] = None, workspace=None):
    """Gradient of the activation from its checkpoint (zq u8 [rows, W], sz f32 [W/128, rows]) and da (f32 or bf16
    [rows, F]): an ActGrad with dzq_cols u8 [rows, W] and sdz_cols f32 [W/128, rows]; with token_tiles dzq_rows u8
    [W, rows] and sdz_rows f32 [rows/128, W]; with recompute aq_rows u8 [F, rows] and sa_rows f32 [rows/128, F]; with
    bias_grad dbias f32 [W]. `out` gives the buffers to write into; what it holds and is not asked for is not written
    and comes back as None."""
    dev = _device(zq)
    rows, W = _dims(zq, "zq", 2)
    if gated and W % 2:
        _fail(f"a gated checkpoint has an even width, got {W}")
    F = W // 2 if gated else W
    _dense(zq, "zq", torch.uint8, (rows, W), dev)
    _dense(sz, "sz", torch.float32, (_cdiv(W, 128), rows), dev)
    ld = _matrix(da, "da", _REAL, (rows, F), dev)
    tiles = _cdiv(rows, 128)
    o = out or (None,) * 7
    qc = _out(o[0], "dzq_cols", torch.uint8, (rows, W), zq, dev)
    sc = _out(o[1], "sdz_cols", torch.float32, (_cdiv(W, 128), rows), zq, dev)
    qr = sr = ar = sa = db = ws = None
    need = 0
    if token_tiles:
        qr = _out(o[2], "dzq_rows", torch.uint8, (W, rows), zq, dev)
        sr = _out(o[3], "sdz_rows", torch.float32, (tiles, W), zq, dev)
    if recompute:
        ar = _out(o[4], "aq_rows", torch.uint8, (F, rows), zq, dev)
        sa = _out(o[5], "sa_rows", torch.float32, (tiles, F), zq, dev)
    if bias_grad:
        db = _out(o[6], "dbias", torch.float32, (W,), zq, dev)
        need = lib().fg_act_checkpoint_bwd_workspace(rows, F, int(bool(gated)))
    if need or workspace is not None:
        ws = _workspace(workspace, need, zq, dev)
    _run("fg_act_checkpoint_bwd", dev, zq.data_ptr(), sz.data_ptr(), da.data_ptr(), _out_code(da.dtype), ld, rows, F,
         _act_code(act), int(bool(gated)), _mode(pow2), qc.data_ptr(), sc.data_ptr(), _addr(qr), _addr(sr), _addr(ar),
         _addr(sa), _addr(db), _addr(ws), 0 if ws is None else ws.numel())
    return ActGrad(qc, sc, qr, sr, ar, sa, db)


def fg_moe_few_tokens(x, ids, weights, w1q, s1, w2q, s2, act: int = FG_ACT_SILU, out_dtype=torch.bfloat16, y=None,
                      pow2: bool = False, workspace=None):
    """A mixture-of-experts feed-forward for at most 64 tokens: x bf16 [T, H], ids int32 and weights f32 [T, topk],
    w1q u8 [E, 2 I, H] (gate rows, then up rows), s1 f32 [E, 2 I/128, H/128], w2q u8 [E, H, I], s2 f32 [E, H/128, I/128]
    -> y [T, H]. Ids outside [0, E) are skipped."""
    dev = _device(x)
    T, H = _dims(x, "x", 2)
    topk = _dims(ids, "ids", 2)[1]
    E, I2, _ = _dims(w1q, "w1q", 3)
    if I2 % 2:
        _fail(f"w1q holds gate and up rows: an even number of them, got {I2}")
    I = I2 // 2
    ld_x = _matrix(x, "x", (torch.bfloat16,), (T, H), dev)
    _dense(ids, "ids", torch.int32, (T, topk), dev)
    _dense(weights, "weights", torch.float32, (T, topk), dev)
    _dense(w1q, "w1q", torch.uint8, (E, I2, H), dev)
    _dense(w2q, "w2q", torch.uint8, (E, H, I), dev)
    if H % 128 == 0 and I % 128 == 0:                # the library refuses others
        _dense(s1, "s1", torch.float32, (E, I2 // 128, H // 128), dev)
        _dense(s2, "s2", torch.float32, (E, H // 128, I // 128), dev)
    if y is None:
        y = torch.empty((T, H), dtype=out_dtype, device=x.device)
    ld_y = _matrix(y, "y", _REAL, (T, H), dev)
    ws = _workspace(workspace, lib().fg_moe_few_tokens_workspace(T, topk, H, I), x, dev)
    _run("fg_moe_few_tokens", dev, x.data_ptr(), ld_x, ids.data_ptr(), weights.data_ptr(), T, topk, w1q.data_ptr(),
         _addr(s1), w2q.data_ptr(), _addr(s2), E, H, I, _act_code(act), _mode(pow2), ws.data_ptr(), ws.numel(),
         y.data_ptr(), ld_y, _out_code(y.dtype))
    return y
