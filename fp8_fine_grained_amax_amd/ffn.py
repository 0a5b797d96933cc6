"""Feed-forward operators (include/fp8fg_ffn.h): the functions carry the C names, check their tensors, allocate outputs
and workspaces the caller does not pass, and run on torch's current stream of the tensors' own device, whichever
device is current. The work of the binding is in the compiled module _ffn (csrc/ffn_binding.cpp)."""
import ctypes
import os
from typing import NamedTuple, Optional

import torch

from . import Fp8fgError, _out_code, lib

FG_ACT_NONE, FG_ACT_RELU, FG_ACT_GELU_TANH, FG_ACT_SILU = 0, 1, 2, 3

_module = None


def _ffn():
    global _module
    if _module is None:
        lib()                                        # fails loudly if the kernels are not built
        try:
            from . import _ffn as module
        except ImportError as e:
            raise Fp8fgError(f"the compiled binding {os.path.join(os.path.dirname(__file__), '_ffn.so')} does not load "
                             f"({e}); run fp8_fine_grained_amax_amd/build.py") from e
        module.set_error(Fp8fgError)
        _module = module
    return _module


def declare(L):
    """Argument types of the feed-forward entry points, for callers of the C library through ctypes."""
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


def fg_fp8_gemm_fprop_epilogue(xq, sx, wq, sw, bias=None, act: int = FG_ACT_NONE, residual=None, out_dtype=torch.bfloat16,
                               y=None, pow2: bool = False):
    """Y [M, N] = act(X [M, K] . W [N, K]^T + bias [N]) + residual [M, N] from E4M3 codes and their scales. bias and
    residual: float32 or bfloat16; residual may have a row stride, and may be y itself."""
    return _ffn().linear(xq, sx, wq, sw, bias, act, residual, _out_code(out_dtype), y, pow2)


def fg_act_checkpoint_fwd(z, act: int, gated: bool = False, pow2: bool = False, zq=None, sz=None, aq=None, sa=None):
    """a = act(z), or act(gate) * up with z = [gate | up], from bf16 z [rows, W]: returns (zq u8 [rows, W], sz f32
    [W/128, rows], aq u8 [rows, F], sa f32 [F/128, rows]), the checkpoint of z and a, both in 1x128 tiles along the
    columns. F = W / 2 when gated, else W."""
    return _ffn().act_forward(z, act, gated, pow2, zq, sz, aq, sa)


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
    return ActGrad._make(_ffn().act_backward(zq, sz, da, act, gated, pow2, token_tiles, recompute, bias_grad, out, workspace))


def fg_moe_few_tokens(x, ids, weights, w1q, s1, w2q, s2, act: int = FG_ACT_SILU, out_dtype=torch.bfloat16, y=None,
                      pow2: bool = False, workspace=None):
    """A mixture-of-experts feed-forward for at most 64 tokens: x bf16 [T, H], ids int32 and weights f32 [T, topk],
    w1q u8 [E, 2 I, H] (gate rows, then up rows), s1 f32 [E, 2 I/128, H/128], w2q u8 [E, H, I], s2 f32 [E, H/128, I/128]
    -> y [T, H]. Ids outside [0, E) are skipped."""
    return _ffn().moe(x, ids, weights, w1q, s1, w2q, s2, act, _out_code(out_dtype), y, pow2, workspace)
