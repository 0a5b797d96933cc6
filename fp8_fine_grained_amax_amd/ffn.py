"""Binding of the feed-forward operators (include/fp8fg_ffn.h): the functions carry the C names, check their
tensors, allocate outputs and workspaces the caller does not pass, and run on torch's current stream of the
tensors' own device, whichever device is current."""
import ctypes
from typing import NamedTuple, Optional

import torch

from . import Fp8fgError, _check, _gpu, _mode, _out_code, _ptr, _stream, lib

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


def _dense(t, what, dtype, shape, device):
    """A contiguous tensor of this type, shape and device."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        _fail(f"{what} must be a contiguous {str(dtype).replace('torch.', '')} tensor of shape {tuple(shape)}, got "
              f"{str(t.dtype).replace('torch.', '')} {tuple(t.shape)} with strides {t.stride()}")
    if t.device != device:
        _fail(f"{what} is on {t.device}, the first argument on {device}")
    return t


def _matrix(t, what, dtypes, shape, device):
    """A row-major matrix whose row stride may exceed its width; its row stride. An empty one has any strides."""
    if t.dtype not in dtypes or tuple(t.shape) != tuple(shape):
        _fail(f"{what} must be a {' or '.join(str(d).replace('torch.', '') for d in dtypes)} matrix of shape "
              f"{tuple(shape)}, got {str(t.dtype).replace('torch.', '')} {tuple(t.shape)}")
    if t.device != device:
        _fail(f"{what} is on {t.device}, the first argument on {device}")
    rows, cols = shape
    if t.numel() == 0 or rows == 1:
        if cols > 1 and t.numel() and t.stride(1) != 1:
            _fail(f"{what} must have unit column stride")
        return cols                                  # a single row has no stride between rows
    if (cols > 1 and t.stride(1) != 1) or t.stride(0) < cols:
        _fail(f"{what} must have unit column stride and rows that do not overlap, got strides {t.stride()}")
    return t.stride(0)


def _out(t, what, dtype, shape, device):
    return torch.empty(shape, dtype=dtype, device=device) if t is None else _dense(t, what, dtype, shape, device)


def _act_code(act):
    if act not in (FG_ACT_NONE, FG_ACT_RELU, FG_ACT_GELU_TANH, FG_ACT_SILU):
        _fail(f"unknown activation {act!r}")
    return int(act)


def _dims(t, what, n):
    if t.dim() != n:
        _fail(f"{what} must have {n} dimensions, got {t.dim()}")
    return t.shape


def _workspace(t, need, device):
    if t is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if t.dtype != torch.uint8 or not t.is_contiguous() or t.device != device:
        _fail(f"workspace must be a contiguous uint8 tensor on {device}")
    return t


def _cdiv(a, b):
    return (a + b - 1) // b


def fg_fp8_gemm_fprop_epilogue(xq, sx, wq, sw, bias=None, act: int = FG_ACT_NONE, residual=None, out_dtype=torch.bfloat16,
                               y=None, pow2: bool = False):
    """Y [M, N] = act(X [M, K] . W [N, K]^T + bias [N]) + residual [M, N] from E4M3 codes and their scales. bias and
    residual: float32 or bfloat16; residual may have a row stride, and may be y itself."""
    _gpu(xq, sx, wq, sw, bias, residual, y)
    M, K = _dims(xq, "xq", 2)
    N, dev = _dims(wq, "wq", 2)[0], xq.device
    _dense(xq, "xq", torch.uint8, (M, K), dev)
    _dense(wq, "wq", torch.uint8, (N, K), dev)
    if K % 128 == 0:                                 # the library refuses others
        _dense(sx, "sx", torch.float32, (K // 128, M), dev)
        _dense(sw, "sw", torch.float32, (_cdiv(N, 128), K // 128), dev)
    if bias is not None:
        _dense(bias, "bias", bias.dtype, (N,), dev)
    ld_res = N
    if residual is not None:
        ld_res = _matrix(residual, "residual", (torch.float32, torch.bfloat16), (M, N), dev)
    y = _out(y, "y", out_dtype if y is None else y.dtype, (M, N), dev)
    with torch.cuda.device(dev):
        _check(lib().fg_fp8_gemm_fprop_epilogue(
            _ptr(xq), _ptr(sx), _ptr(wq), _ptr(sw), M, N, K, _ptr(bias), 0 if bias is None else _out_code(bias.dtype),
            _act_code(act), _ptr(residual), 0 if residual is None else _out_code(residual.dtype), ld_res, _ptr(y),
            _out_code(y.dtype), _mode(pow2), _stream(dev)), "fg_fp8_gemm_fprop_epilogue")
    return y


def fg_act_checkpoint_fwd(z, act: int, gated: bool = False, pow2: bool = False, zq=None, sz=None, aq=None, sa=None):
    """a = act(z), or act(gate) * up with z = [gate | up], from bf16 z [rows, W]: returns (zq u8 [rows, W], sz f32
    [W/128, rows], aq u8 [rows, F], sa f32 [F/128, rows]), the checkpoint of z and a, both in 1x128 tiles along the
    columns. F = W / 2 when gated, else W."""
    _gpu(z, zq, sz, aq, sa)
    rows, W = _dims(z, "z", 2)
    if gated and W % 2:
        _fail(f"a gated z has an even width, got {W}")
    F, dev = W // 2 if gated else W, z.device
    ld = _matrix(z, "z", (torch.bfloat16,), (rows, W), dev)
    zq = _out(zq, "zq", torch.uint8, (rows, W), dev)
    sz = _out(sz, "sz", torch.float32, (_cdiv(W, 128), rows), dev)
    aq = _out(aq, "aq", torch.uint8, (rows, F), dev)
    sa = _out(sa, "sa", torch.float32, (_cdiv(F, 128), rows), dev)
    with torch.cuda.device(dev):
        _check(lib().fg_act_checkpoint_fwd(_ptr(z), rows, F, ld, _act_code(act), int(bool(gated)), _mode(pow2), _ptr(zq),
                                           _ptr(sz), _ptr(aq), _ptr(sa), _stream(dev)), "fg_act_checkpoint_fwd")
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
    bias_grad dbias f32 [W]. `out` gives the buffers to write into."""
    _gpu(zq, sz, da, workspace, *(out or ()))
    rows, W = _dims(zq, "zq", 2)
    if gated and W % 2:
        _fail(f"a gated checkpoint has an even width, got {W}")
    F, dev = W // 2 if gated else W, zq.device
    _dense(zq, "zq", torch.uint8, (rows, W), dev)
    _dense(sz, "sz", torch.float32, (_cdiv(W, 128), rows), dev)
    ld = _matrix(da, "da", (torch.float32, torch.bfloat16), (rows, F), dev)
    want = (True, True, token_tiles, token_tiles, recompute, recompute, bias_grad)
    shapes = ((rows, W), (_cdiv(W, 128), rows), (W, rows), (_cdiv(rows, 128), W), (F, rows), (_cdiv(rows, 128), F), (W,))
    types = (torch.uint8, torch.float32) * 3 + (torch.float32,)
    given = out or (None,) * 7
    r = ActGrad(*(_out(t, n, d, s, dev) if w else None
                  for w, t, n, d, s in zip(want, given, ActGrad._fields, types, shapes)))
    need = lib().fg_act_checkpoint_bwd_workspace(rows, F, int(bool(gated))) if bias_grad else 0
    ws = _workspace(workspace, need, dev) if need or workspace is not None else None
    with torch.cuda.device(dev):
        _check(lib().fg_act_checkpoint_bwd(
            _ptr(zq), _ptr(sz), _ptr(da), _out_code(da.dtype), ld, rows, F, _act_code(act), int(bool(gated)), _mode(pow2),
            _ptr(r.dzq_cols), _ptr(r.sdz_cols), _ptr(r.dzq_rows), _ptr(r.sdz_rows), _ptr(r.aq_rows), _ptr(r.sa_rows),
            _ptr(r.dbias), _ptr(ws), 0 if ws is None else ws.numel(), _stream(dev)), "fg_act_checkpoint_bwd")
    return r


def fg_moe_few_tokens(x, ids, weights, w1q, s1, w2q, s2, act: int = FG_ACT_SILU, out_dtype=torch.bfloat16, y=None,
                      pow2: bool = False, workspace=None):
    """A mixture-of-experts feed-forward for at most 64 tokens: x bf16 [T, H], ids int32 and weights f32 [T, topk],
    w1q u8 [E, 2 I, H] (gate rows, then up rows), s1 f32 [E, 2 I/128, H/128], w2q u8 [E, H, I], s2 f32 [E, H/128, I/128]
    -> y [T, H]. Ids outside [0, E) are skipped."""
    _gpu(x, ids, weights, w1q, s1, w2q, s2, y, workspace)
    T, H = _dims(x, "x", 2)
    topk, dev = _dims(ids, "ids", 2)[1], x.device
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
        y = torch.empty((T, H), dtype=out_dtype, device=dev)
    ld_y = _matrix(y, "y", (torch.float32, torch.bfloat16), (T, H), dev)
    ws = _workspace(workspace, lib().fg_moe_few_tokens_workspace(T, topk, H, I), dev)
    with torch.cuda.device(dev):
        _check(lib().fg_moe_few_tokens(
            _ptr(x), ld_x, _ptr(ids), _ptr(weights), T, topk, _ptr(w1q), _ptr(s1), _ptr(w2q), _ptr(s2), E, H, I,
            _act_code(act), _mode(pow2), _ptr(ws), ws.numel(), _ptr(y), ld_y, _out_code(y.dtype), _stream(dev)),
            "fg_moe_few_tokens")
    return y
