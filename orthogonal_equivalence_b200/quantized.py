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

from typing import NamedTuple, Optional, Tuple

import torch

from . import (POETX_BF16, POETX_FP32, _check, lib, poetx_block_backward_workspace_bytes,
               poetx_matmul_int8_grad_workspace_bytes, poetx_matmul_int8_workspace_bytes,
               poetx_rmsnorm_backward_workspace_bytes)

_DTYPE = {torch.bfloat16: POETX_BF16, torch.float32: POETX_FP32}


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


def _like(t, name: str, dtype=None, shape=None, device=None) -> None:
    """Host-side check of a tensor before its pointer goes to the library."""
    try:  # the good case, at the cost of a few attribute reads
        if ((dtype is None or t.dtype == dtype) and (shape is None or t.shape == shape)
                and (device is None or t.device == device) and t.is_contiguous()):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: tensor on {t.device}, the other operands are on {device}")
    raise ValueError(f"{name}: must be contiguous")


def _rows(t, name: str) -> Tuple[int, int]:
    """T, d of a contiguous 2-D activation in a dtype of the library."""
    _like(t, name)
    if t.dtype not in _DTYPE:
        raise ValueError(f"{name}: dtype {t.dtype}, expected torch.bfloat16 or torch.float32")
    shape = t.shape
    if len(shape) != 2 or shape[1] == 0:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [T][d] with d >= 1")
    return shape


def _codes(t, name: str) -> Tuple[int, int]:
    _like(t, name, torch.int8)
    shape = t.shape
    if len(shape) != 2 or shape[1] == 0:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [rows][d] with d >= 1")
    return shape


_calls = {}


def _run(device: torch.device, fn: str, *args) -> None:
    """The C call on the current stream of `device`, with that device current."""
    if device.type != "cuda":
        raise ValueError(f"tensors on {device}: the library runs on CUDA devices")
    call = _calls.get(fn)
    if call is None:
        call = _calls[fn] = getattr(lib(), fn)
    index = device.index
    if index == torch.cuda.current_device():
        status = call(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = call(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _check(status, fn)


def _p(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def quantize_rows(x: torch.Tensor, colscale: Optional[torch.Tensor] = None) -> QuantRows:
    """Rows of x (or of x * colscale, colscale fp32 [d]) as int8 codes with one scale per row."""
    T, d = _rows(x, "x")
    dev = x.device
    if colscale is not None:
        _like(colscale, "colscale", torch.float32, (d,), dev)
    out = QuantRows(torch.empty_like(x, dtype=torch.int8),
                    torch.empty(T, dtype=torch.float32, device=dev))
    _run(dev, "poetx_quantize_rows", T, d, x.data_ptr(), _DTYPE[x.dtype], _p(colscale), out.codes.data_ptr(),
         out.scale.data_ptr())
    return out


def dequantize_rows(codes: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """codes * scale per row, rounded once to dtype (the weight dequantiser on any rows)."""
    T, d = _codes(codes, "codes")
    dev = codes.device
    _like(scale, "scale", torch.float32, (T,), dev)
    if dtype not in _DTYPE:
        raise ValueError(f"dtype: {dtype}, expected torch.bfloat16 or torch.float32")
    out = torch.empty_like(codes, dtype=dtype)
    _run(dev, "poetx_weight_dequantize", T, d, codes.data_ptr(), scale.data_ptr(), _DTYPE[dtype], out.data_ptr())
    return out


def rmsnorm_quantize(x: torch.Tensor, gamma: torch.Tensor, residual: Optional[torch.Tensor] = None,
                     eps: float = 1e-5, codes: bool = True, y: bool = False) -> NormRows:
    """h = x + residual and its root-mean-square norm with gain gamma (fp32
    [d]), as int8 rows (`codes`) and / or in x's dtype (`y`)."""
    T, d = _rows(x, "x")
    dev, dt = x.device, x.dtype
    _like(gamma, "gamma", torch.float32, (d,), dev)
    h = None
    if residual is not None:
        _like(residual, "residual", dt, x.shape, dev)
        h = torch.empty_like(x)
    q = torch.empty_like(x, dtype=torch.int8) if codes else None
    s = gamma.new_empty(T) if codes else None
    out = torch.empty_like(x) if y else None
    rstd = gamma.new_empty(T)
    _run(dev, "poetx_rmsnorm_quantize", T, d, x.data_ptr(), _p(residual), gamma.data_ptr(), eps, _DTYPE[dt], _p(h),
         _p(out), _p(q), _p(s), rstd.data_ptr())
    return NormRows(q, s, x if h is None else h, rstd, out)


def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor,
                     dres: Optional[torch.Tensor] = None,
                     dgamma: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dgamma) of the norm from the gradient dy of its rows and, with
    dres, the gradient that reaches h past it; dx is the gradient of x and of
    the residual.  A dgamma that is handed in is added to."""
    T, d = _rows(dy, "dy")
    dev, dt = dy.device, dy.dtype
    _like(h, "h", dt, dy.shape, dev)
    _like(gamma, "gamma", torch.float32, (d,), dev)
    _like(rstd, "rstd", torch.float32, (T,), dev)
    if dres is not None:
        _like(dres, "dres", dt, dy.shape, dev)
    accumulate = dgamma is not None
    if accumulate:
        _like(dgamma, "dgamma", torch.float32, (d,), dev)
    else:
        dgamma = torch.empty_like(gamma)
    dx = torch.empty_like(dy)
    nb = poetx_rmsnorm_backward_workspace_bytes(T, d, _DTYPE[dt])
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    _run(dev, "poetx_rmsnorm_backward", T, d, dy.data_ptr(), h.data_ptr(), gamma.data_ptr(), rstd.data_ptr(),
         _p(dres), _DTYPE[dt], dx.data_ptr(), dgamma.data_ptr(), int(accumulate), ws.data_ptr(), nb)
    return dx, dgamma


def matmul_int8(xq: torch.Tensor, xscale: torch.Tensor, Wq: torch.Tensor, wscale: torch.Tensor,
                dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """z[t][j] = xscale[t] wscale[j] sum_i xq[t][i] Wq[j][i] in dtype, the sum exact."""
    T, m = _codes(xq, "xq")
    dev = xq.device
    n, _ = _codes(Wq, "Wq")
    if Wq.shape[1] != m or Wq.device != dev:
        _like(Wq, "Wq", torch.int8, (n, m), dev)
    _like(xscale, "xscale", torch.float32, (T,), dev)
    _like(wscale, "wscale", torch.float32, (n,), dev)
    if dtype not in _DTYPE:
        raise ValueError(f"dtype: {dtype}, expected torch.bfloat16 or torch.float32")
    out = torch.empty(T, n, dtype=dtype, device=dev)
    nb, ws = 0, None
    if m % 16:  # rows that are no whole 16-byte units are copied first
        nb = poetx_matmul_int8_workspace_bytes(T, n, m)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    _run(dev, "poetx_matmul_int8", T, n, m, xq.data_ptr(), xscale.data_ptr(), Wq.data_ptr(), wscale.data_ptr(),
         _DTYPE[dtype], out.data_ptr(), _p(ws), nb)
    return out


def matmul_int8_grad(dz: torch.Tensor, Wq: torch.Tensor, wscale: torch.Tensor) -> torch.Tensor:
    """dx of matmul_int8's tokens from dz, in dz's dtype: dz * wscale quantised
    row by row, times Wq over the channels."""
    T, n = _rows(dz, "dz")
    dev = dz.device
    _, m = _codes(Wq, "Wq")
    if Wq.shape[0] != n or Wq.device != dev:
        _like(Wq, "Wq", torch.int8, (n, m), dev)
    _like(wscale, "wscale", torch.float32, (n,), dev)
    dx = torch.empty(T, m, dtype=dz.dtype, device=dev)
    nb = poetx_matmul_int8_grad_workspace_bytes(T, n, m)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    _run(dev, "poetx_matmul_int8_grad", T, n, m, dz.data_ptr(), Wq.data_ptr(), wscale.data_ptr(), _DTYPE[dz.dtype],
         dx.data_ptr(), ws.data_ptr(), nb)
    return dx


def checkpoint_save(x: torch.Tensor) -> Checkpoint:
    """x as int8 codes with a shared power of two per 32 columns."""
    T, d = _rows(x, "x")
    dev = x.device
    out = Checkpoint(torch.empty_like(x, dtype=torch.int8),
                     torch.empty(T, (d + 31) // 32, dtype=torch.uint8, device=dev))
    _run(dev, "poetx_checkpoint_save", T, d, x.data_ptr(), _DTYPE[x.dtype], out.codes.data_ptr(),
         out.exps.data_ptr())
    return out


def _checkpoint(c: Checkpoint, name: str) -> Tuple[int, int]:
    T, d = _codes(c.codes, f"{name} codes")
    _like(c.exps, f"{name} exps", torch.uint8, (T, (d + 31) // 32), c.codes.device)
    return T, d


def checkpoint_load(ckpt: Checkpoint, dtype: torch.dtype) -> torch.Tensor:
    """The values a checkpoint stands for (exact in both dtypes)."""
    T, d = _checkpoint(ckpt, "checkpoint")
    if dtype not in _DTYPE:
        raise ValueError(f"dtype: {dtype}, expected torch.bfloat16 or torch.float32")
    dev = ckpt.codes.device
    out = torch.empty_like(ckpt.codes, dtype=dtype)
    _run(dev, "poetx_checkpoint_load", T, d, ckpt.codes.data_ptr(), ckpt.exps.data_ptr(), _DTYPE[dtype],
         out.data_ptr())
    return out


def block_backward(ckpt: Checkpoint, D: torch.Tensor, G: torch.Tensor, need_o: bool = True,
                   dG: Optional[torch.Tensor] = None) -> Tuple[Optional[torch.Tensor], torch.Tensor]:
    """(O, dG) of one side of a layer from its activation's checkpoint X:
    O_j = D_j G_j^T and dG_j = X_j^T D_j (fp32).  A dG that is handed in is
    added to."""
    T, d = _checkpoint(ckpt, "checkpoint")
    dev = ckpt.codes.device
    _rows(D, "D")
    _like(D, "D", None, (T, d), dev)
    if not isinstance(G, torch.Tensor) or G.dim() != 3 or G.shape[0] == 0 or d % G.shape[0]:
        raise ValueError(f"G: expected [d/b][b][b] with d = {d}")
    b = d // G.shape[0]
    _like(G, "G", D.dtype, (d // b, b, b), dev)
    accumulate = dG is not None
    if accumulate:
        _like(dG, "dG", torch.float32, G.shape, dev)
    else:
        dG = torch.empty(d // b, b, b, dtype=torch.float32, device=dev)
    O = torch.empty_like(D) if need_o else None
    dt = _DTYPE[D.dtype]
    nb = poetx_block_backward_workspace_bytes(T, d, b, dt)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    _run(dev, "poetx_block_backward", T, d, b, ckpt.codes.data_ptr(), ckpt.exps.data_ptr(), D.data_ptr(),
         G.data_ptr(), dt, _p(O), dG.data_ptr(), int(accumulate), ws.data_ptr(), nb)
    return O, dG
