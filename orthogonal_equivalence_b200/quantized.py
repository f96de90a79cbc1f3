"""The 8-bit path on torch tensors: rows quantised to int8, the norm that ends
in such rows, the int8 product with the POET-XQ weight and its gradient, and
activation checkpoints with the block backward that reads them.  Allocation
and checks here, arithmetic in libpoetx.so (include/poetx.h states each
operator's formula).

Every call runs on the current stream of its tensors' device and allocates its
outputs and workspace there with torch, so calls of one stream may be captured
into a CUDA graph (each capture holds its own workspace).  Tensors used on
another stream than the one they were made on follow torch's own rule
(Tensor.record_stream).  These functions are not recorded by autograd: the
backward of each is a call of its own.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from . import SIGNATURES, _check, lib

_native = None


def native():
    """The extension _tensors.so (csrc/tensors.cpp: argument checks, outputs
    from torch's allocator, the C call), bound to the loaded libpoetx.so."""
    global _native
    if _native is None:
        L = lib()
        try:
            from . import _tensors
        except ImportError as e:
            raise RuntimeError(f"_tensors.so not built or not loadable ({e}); run orthogonal_equivalence_b200/build.py")
        _tensors.bind({name: ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in SIGNATURES}, _check,
                      torch.OutOfMemoryError)
        _native = _tensors
    return _native


class QuantRows(NamedTuple):
    """Rows as int8 codes [T][d] and one fp32 scale per row: row = codes * scale."""
    codes: torch.Tensor
    scale: torch.Tensor


class NormRows(NamedTuple):
    """What rmsnorm_quantize returns: the normalised rows (codes, scale), h = x
    + residual and rstd for the backward, and y, the rows in x's dtype, if asked."""
    codes: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    h: torch.Tensor
    rstd: torch.Tensor
    y: Optional[torch.Tensor]


class Checkpoint(NamedTuple):
    """An activation [T][d] kept in 8 bits: int8 codes and one biased exponent
    (uint8) per 32 columns."""
    codes: torch.Tensor
    exps: torch.Tensor


def quantize_rows(x: torch.Tensor, colscale: Optional[torch.Tensor] = None) -> QuantRows:
    """Rows of x (or of x * colscale, colscale fp32 [d]) as int8 codes with one scale per row."""
    return QuantRows(*native().quantize_rows(x, colscale))


def dequantize_rows(codes: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """codes * scale per row, rounded once to dtype (the weight dequantiser on any rows)."""
    return native().dequantize_rows(codes, scale, dtype)


def rmsnorm_quantize(x: torch.Tensor, gamma: torch.Tensor, residual: Optional[torch.Tensor] = None,
                     eps: float = 1e-5, codes: bool = True, y: bool = False) -> NormRows:
    """h = x + residual and its root-mean-square norm with gain gamma (fp32
    [d]), as int8 rows (`codes`) and / or in x's dtype (`y`)."""
    return NormRows(*native().rmsnorm_quantize(x, gamma, residual, eps, codes, y))


def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor,
                     dres: Optional[torch.Tensor] = None,
                     dgamma: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dgamma) of the norm from the gradient dy of its rows and, with
    dres, the gradient that reaches h past it; dx is the gradient of x and of
    the residual.  A dgamma that is handed in is added to."""
    return native().rmsnorm_backward(dy, h, gamma, rstd, dres, dgamma)


def matmul_int8(xq: torch.Tensor, xscale: torch.Tensor, Wq: torch.Tensor, wscale: torch.Tensor,
                dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """z[t][j] = xscale[t] wscale[j] sum_i xq[t][i] Wq[j][i] in dtype, the sum exact."""
    return native().matmul_int8(xq, xscale, Wq, wscale, dtype)


def matmul_int8_grad(dz: torch.Tensor, Wq: torch.Tensor, wscale: torch.Tensor) -> torch.Tensor:
    """dx of matmul_int8's tokens from dz, in dz's dtype: dz * wscale quantised
    row by row, times Wq over the channels."""
    return native().matmul_int8_grad(dz, Wq, wscale)


def checkpoint_save(x: torch.Tensor) -> Checkpoint:
    """x as int8 codes with a shared power of two per 32 columns."""
    return Checkpoint(*native().checkpoint_save(x))


def checkpoint_load(ckpt: Checkpoint, dtype: torch.dtype) -> torch.Tensor:
    """The values a checkpoint stands for (exact in both dtypes)."""
    return native().checkpoint_load(ckpt.codes, ckpt.exps, dtype)


def block_backward(ckpt: Checkpoint, D: torch.Tensor, G: torch.Tensor, need_o: bool = True,
                   dG: Optional[torch.Tensor] = None) -> Tuple[Optional[torch.Tensor], torch.Tensor]:
    """(O, dG) of one side of a layer from its activation's checkpoint X:
    O_j = D_j G_j^T and dG_j = X_j^T D_j (fp32).  A dG that is handed in is
    added to."""
    return native().block_backward(ckpt.codes, ckpt.exps, D, G, need_o, dG)
