"""The two ends of a Linear's training step (include/fp8fg_train.h): the norm whose output is the Linear's FP8 operand, its
backward pass, and the orthogonalised update of the weight. The functions carry the C names, check their tensors, allocate
outputs and workspaces the caller does not pass, and run on torch's current stream of the tensors' own device,
whichever device is current. The work of the binding is in the compiled module _ffn (csrc/train_binding.cpp)."""
import ctypes
from typing import NamedTuple, Optional

import torch

from . import _out_code
from .ffn import _ffn

FG_NORM_LAYER, FG_NORM_RMS = 0, 1


def declare(L):
    """Argument types of these entry points, for callers of the C library through ctypes."""
    P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    L.fg_norm_quantize.argtypes = [P, I, I64, I64, I64, I, P, P, I, F, I, P, P, P, P, P, P, P, P]
    L.fg_norm_bwd.argtypes = [P, I, I64, P, P, P, I, P, I, I64, P, I, I64, I64, I64, I, P, I, P, P, I, P, I64, P]
    L.fg_orthogonalize.argtypes = [P, I, I64, I64, I64, I64, I, F, F, F, F, F, P, P, I64, P]
    for f in ("fg_norm_quantize", "fg_norm_bwd", "fg_orthogonalize"):
        getattr(L, f).restype = I
    L.fg_norm_bwd_workspace.argtypes = [I64, I64]
    L.fg_orthogonalize_workspace.argtypes = [I64, I64, I64]
    for f in ("fg_norm_bwd_workspace", "fg_orthogonalize_workspace"):
        getattr(L, f).restype = I64


class NormTiles(NamedTuple):
    """What fg_norm_quantize returns: y in tiles along the columns (the Fprop's operand), along the rows (the Wgrad's) and in
    bf16, and the statistics of the rows; None for what was not asked for."""
    q_cols: torch.Tensor
    s_cols: torch.Tensor
    q_rows: Optional[torch.Tensor]
    s_rows: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    mean: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


_NO_TILES = NormTiles(*[None] * 7)


def fg_norm_quantize(x, gamma, beta=None, kind: int = FG_NORM_LAYER, eps: float = 1e-5, pow2: bool = False,
                     token_tiles: bool = False, with_y: bool = False, statistics: bool = True,
                     out: Optional[NormTiles] = None):
    """Layer or RMS norm of each row of x (f32 or bf16 [rows, cols]), y = (x - mean) rstd gamma + beta (RMS: x rstd gamma +
    beta), as FP8 tiles: a NormTiles with q_cols u8 [rows, cols] and s_cols f32 [cols/128, rows]; with token_tiles q_rows u8
    [cols, rows] and s_rows f32 [rows/128, cols]; with with_y y bf16; with statistics or token_tiles mean (layer norm) and
    rstd f32 [rows]. gamma and beta: f32 or bf16 [cols]. `out` gives the buffers to write into; what it holds and is not
    asked for is not written and comes back as None."""
    return NormTiles._make(_ffn().norm_quantize(x, gamma, beta, kind, eps, pow2, token_tiles, with_y, statistics,
                                                *(_NO_TILES if out is None else out)))


class NormGrad(NamedTuple):
    """What fg_norm_bwd returns; None for what was not asked for."""
    dx: torch.Tensor
    dgamma: Optional[torch.Tensor]
    dbeta: Optional[torch.Tensor]


def fg_norm_bwd(x, mean, rstd, gamma, dy, residual_grad=None, kind: int = FG_NORM_LAYER, out_dtype=torch.bfloat16,
                weight_grad: bool = True, bias_grad: bool = False, accumulate: bool = False, dx=None, dgamma=None, dbeta=None,
                workspace=None):
    """Backward of fg_norm_quantize's norm: dx [rows, cols] (out_dtype) from dy (f32 or bf16 [rows, cols]), plus
    residual_grad where it is given (it may be dx itself); with weight_grad dgamma and with bias_grad dbeta, f32 [cols], added
    to what dgamma and dbeta hold with accumulate."""
    return NormGrad._make(_ffn().norm_bwd(x, mean, rstd, gamma, dy, residual_grad, kind, _out_code(out_dtype), weight_grad,
                                          bias_grad, accumulate, dx, (dgamma, dbeta), workspace))


def fg_orthogonalize(g, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, scale: float = 1.0, out=None,
                     workspace=None):
    """Orthogonalised update by Newton-Schulz products: of each matrix of g (f32 or bf16, [N, K] or [batch, N, K]), X = g / (|g| +
    eps), `steps` times X = (a I + b A + c A A) X with A = X X^T, and scale X as bf16. X, A and the sum in brackets are held in fp16;
    fp8fg_train.h says how exact that leaves updates of gradients with different spectra."""
    a, b, c = coefficients
    return _ffn().orthogonalize(g, steps, a, b, c, eps, scale, out, workspace)
