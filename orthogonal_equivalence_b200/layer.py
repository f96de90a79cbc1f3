"""PoetxLinear: device buffers of one POET-X layer and thin wrappers around
the C calls (allocation with torch, arithmetic in libpoetx.so).

State of a layer (POET-X write-up, sections 2-3 and the merge step of its API
snippet): the frozen weight stored in the frame of the current permutations
(W[j'][i'] = W0[permR[i']][permP[j']], [n][m]), the permutations, the packed
triangles qR, qP (the trainable parameters) and the G blocks built from them.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import (POETX_BF16, POETX_FOLD_ALL, POETX_FP32, make_layer, poetx_backward, poetx_backward_dG,
               poetx_backward_recompute_workspace_bytes, poetx_backward_workspace_bytes, poetx_cnp_backward,
               poetx_cnp_workspace_bytes,
               poetx_forward, poetx_forward_workspace_bytes, poetx_frame_export, poetx_frame_import,
               poetx_layer_cnp_build, poetx_layer_cnp_workspace_bytes, poetx_layers_cnp_build,
               poetx_layers_cnp_workspace_bytes, poetx_merge, poetx_merge_workspace_bytes, poetx_weight_dequantize,
               poetx_weight_quantize, poetx_adamw_step, make_q8, poetx_forward_q8, poetx_forward_q8_workspace_bytes,
               poetx_backward_q8, poetx_backward_dG_q8, poetx_backward_q8_workspace_bytes)
from .quantized import Checkpoint, matmul_int8, matmul_int8_grad, quantize_rows

_TORCH_DTYPE = {POETX_BF16: torch.bfloat16, POETX_FP32: torch.float32}


def _need(t, shape, dtype, device: torch.device, name: str) -> None:
    """Host-side check of a tensor handed to the library.  The C calls take
    raw device pointers and trust the layer's sizes, so a tensor of another
    shape, dtype, device or stride must be refused here, before any launch."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device.type != device.type or (device.index is not None and t.device.index != device.index):
        raise ValueError(f"{name}: tensor on {t.device}, the layer is on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _torch_stream(stream, device: torch.device):
    """The torch stream of a call's `stream` argument (a stream or its handle); None where none is given."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    return torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)


def _on(stream, device: torch.device):
    """A context in which `device` is the current one and torch's own work and
    allocations belong to the stream a call is given (the device's current one
    where it is given none): the C calls run on the current device."""
    if device.type != "cuda":
        return contextlib.nullcontext()
    s = _torch_stream(stream, device)
    return torch.cuda.device(device) if s is None else torch.cuda.stream(s)


def _drop(t: torch.Tensor, stream) -> None:
    """`t` is let go while a call on `stream` may still read it."""
    if stream is not None and t.device.type == "cuda":
        t.record_stream(_torch_stream(stream, t.device))


def _workspace(held: dict, kind: str, nbytes: int, device: torch.device, stream=None) -> torch.Tensor:
    """Scratch of a call on `stream`: held and reused by eager calls (which are
    therefore to be ordered on one stream), but a captured call's own, from its
    graph's memory, so that no two graphs share it and no later eager call that
    needs more can free it under a graph.  It is allocated on the call's
    stream, which is therefore the only one that can get its memory next."""
    with _on(stream, device):
        if device.type == "cuda" and torch.cuda.is_current_stream_capturing():
            return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
        ws = held.get(kind)
        if ws is None or ws.numel() < nbytes:
            ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
            held[kind] = ws
        return ws


class Saved(NamedTuple):
    """Activations the forward keeps for the backward: Y ([T][n], the P-side
    input in the Psi_P frame) and optionally Xg ([T][m], x in the Psi_R frame),
    as tensors of the layer dtype or as 8-bit checkpoints (forward(save8=True))."""
    y: Union[torch.Tensor, Checkpoint, None]
    xg: Union[torch.Tensor, Checkpoint, None]


class PoetxLinear:
    """One layer z = x R W0 P (x: [T][m], z: [T][n]).

    `fold` (POETX_FOLD_* bits, default 0) lets a bf16 layer apply a block
    product to the weight instead of the token rows where that moves fewer
    bytes; 0 keeps the write-up's input-centric evaluation everywhere."""

    def __init__(self, m: int, n: int, b: int, dtype: int, device="cuda", fold: int = 0):
        if dtype not in _TORCH_DTYPE:
            raise ValueError("dtype must be POETX_BF16 or POETX_FP32")
        if fold & ~POETX_FOLD_ALL:
            raise ValueError("fold: unknown POETX_FOLD bits")
        self.fold = fold
        self.m, self.n, self.b, self.dtype = m, n, b, dtype
        self.device = torch.device(device)
        td = _TORCH_DTYPE[dtype]
        tri = b * (b - 1) // 2
        self.W = torch.empty((n, m), dtype=td, device=self.device)
        self.permR = torch.empty(m, dtype=torch.int32, device=self.device)
        self.permP = torch.empty(n, dtype=torch.int32, device=self.device)
        self.qR = torch.zeros((m // b, tri), dtype=torch.float32, device=self.device)
        self.qP = torch.zeros((n // b, tri), dtype=torch.float32, device=self.device)
        self.GR = torch.empty((m // b, b, b), dtype=td, device=self.device)
        self.GP = torch.empty((n // b, b, b), dtype=td, device=self.device)
        self._ws = {}
        self.Wq = None      # POET-XQ: int8 codes of W and per-row scales
        self.Wscale = None
        self._wscratch = None
        self.int8_product = False

    # -------------------------------------------------------------- POET-XQ
    def quantize_weight(self, scratch: Optional[torch.Tensor] = None, stream=None, int8_product: bool = False) -> None:
        """Keep W as int8 codes + per-row scales (POET-XQ) and drop the bf16
        copy; every forward / backward dequantizes it into `scratch` (a flat
        tensor of at least n*m elements of the layer dtype, which several
        layers may share) right before use.  With `int8_product` there is no
        scratch: the W0 product of the forward and of the backward multiplies
        the codes themselves with its other operand quantized row by row (see
        poetx_q8 in include/poetx.h); merge and export need the weight and
        refuse then.  A layer that already has codes keeps them: the call only
        changes how they are used."""
        self._need_weight("quantize_weight")
        if int8_product and self.fold:
            raise ValueError("int8_product: the layer folds its blocks into the weight (fold != 0)")
        if int8_product and scratch is not None:
            raise ValueError("scratch: not used with int8_product")
        if not int8_product:
            if scratch is None:
                scratch = torch.empty(self.n * self.m, dtype=self.torch_dtype, device=self.device)
            if scratch.numel() < self.n * self.m:
                raise ValueError(f"scratch: {scratch.numel()} elements, the layer needs {self.n * self.m}")
            _need(scratch, (scratch.numel(),), self.torch_dtype, self.device, "scratch")
        if self.Wq is None:  # (else W is the scratch, which holds any layer's weight or none)
            Wq = torch.empty((self.n, self.m), dtype=torch.int8, device=self.device)
            Wscale = torch.empty(self.n, dtype=torch.float32, device=self.device)
            with self._on(stream):
                poetx_weight_quantize(self.n, self.m, self.W, self.dtype, Wq, Wscale, stream)
            _drop(self.W, stream)
            self.Wq, self.Wscale = Wq, Wscale
        self.int8_product = int8_product
        self._wscratch = scratch
        # (int8_product: W stands for the pointer only, no call of this mode reads it)
        self.W = self.Wq if int8_product else scratch[: self.n * self.m].view(self.n, self.m)

    def _dequantize(self, stream=None) -> None:
        if self.Wq is not None and not self.int8_product:
            self.W = self._wscratch[: self.n * self.m].view(self.n, self.m)
            poetx_weight_dequantize(self.n, self.m, self.Wq, self.Wscale, self.dtype, self.W, stream)

    @property
    def torch_dtype(self) -> torch.dtype:
        return _TORCH_DTYPE[self.dtype]

    def abi(self):
        self._need_weight("abi")
        return self._abi()

    def _abi(self):
        return make_layer(self.m, self.n, self.b, self.dtype, self.W, self.permR, self.permP, self.qR, self.qP,
                          self.GR, self.GP, self.fold)

    def _on(self, stream):
        return _on(stream, self.permR.device)

    def workspace(self, kind: str, nbytes: int, stream=None) -> torch.Tensor:
        return _workspace(self._ws, kind, nbytes, self.device, stream)

    # -------------------------------------------------------------- state
    def load(self, W0lin: torch.Tensor, permR: torch.Tensor, permP: torch.Tensor, qR: torch.Tensor,
             qP: torch.Tensor, stream=None) -> None:
        """Set the permutations and triangles, import the natural nn.Linear
        weight W0^T ([n][m]) into the frame, and build G.  A layer that kept
        its weight as codes is one with its weight in full again."""
        with self._on(stream):
            W0lin = W0lin.contiguous()
        _need(W0lin, (self.n, self.m), self.torch_dtype, self.device, "W0lin")
        for name, t, shape in (("permR", permR, self.permR.shape), ("permP", permP, self.permP.shape),
                               ("qR", qR, self.qR.shape), ("qP", qP, self.qP.shape)):
            if tuple(t.shape) != tuple(shape):
                raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if self.Wq is not None:  # W is the codes, or a scratch that the old codes would be expanded into
            self.W = torch.empty((self.n, self.m), dtype=self.torch_dtype, device=self.device)
            self.Wq = self.Wscale = self._wscratch = None
            self.int8_product = False
        with self._on(stream):
            self.permR.copy_(permR)
            self.permP.copy_(permP)
            self.qR.copy_(qR)
            self.qP.copy_(qP)
            poetx_frame_import(self.abi(), W0lin, stream)
        self.build(stream)

    def _need_weight(self, what: str) -> None:
        if self.int8_product:
            raise RuntimeError(f"{what}: the layer keeps its weight as int8 codes only (int8_product)")

    def _q8(self, y, xg):
        """The poetx_q8 of a call with these saved activations, or None."""
        y8, xg8 = isinstance(y, Checkpoint), isinstance(xg, Checkpoint)
        if not (y8 or xg8 or self.int8_product):
            return None
        return make_q8(self.Wq if self.int8_product else None, self.Wscale if self.int8_product else None,
                       y.codes if y8 else None, y.exps if y8 else None, xg.codes if xg8 else None,
                       xg.exps if xg8 else None)

    def _new_checkpoint(self, T: int, d: int) -> Checkpoint:
        return Checkpoint(torch.empty((T, d), dtype=torch.int8, device=self.device),
                          torch.empty((T, (d + 31) // 32), dtype=torch.uint8, device=self.device))

    def export_weight(self, stream=None) -> torch.Tensor:
        self._need_weight("export_weight")
        out = torch.empty((self.n, self.m), dtype=self.torch_dtype, device=self.device)
        with self._on(stream):
            self._dequantize(stream)
            poetx_frame_export(self.abi(), out, stream)
        return out

    def build(self, stream=None) -> None:
        """G_R, G_P from qR, qP (Cayley-Neumann), both sides in one batch."""
        with self._on(stream):
            L = self._abi()
            nb = poetx_layer_cnp_workspace_bytes(L)
            ws = self.workspace("cnp", nb, stream)
            poetx_layer_cnp_build(L, ws, nb, stream)

    # -------------------------------------------------------------- layer
    def forward(self, x: torch.Tensor, save: bool = True, save_xg: bool = False, z: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None, xg: Optional[torch.Tensor] = None,
                stream=None, save8: bool = False) -> Tuple[torch.Tensor, Optional["Saved"]]:
        """z = x R W0 P.  With `save`, also returns what the backward needs:
        Y (the P-side input) and, with `save_xg`, Xg = x[:, permR].  With
        `save8` both are kept as 8-bit checkpoints (int8 codes and an exponent
        per 32 columns, about half the bytes; y and xg, if given, are
        Checkpoints to write into): z is the same, and so is the backward's
        dx, while the gradients of the triangles see the checkpoints' values."""
        T = x.shape[0]
        td = self.torch_dtype
        _need(x, (T, self.m), td, self.device, "x")
        if z is None:
            z = torch.empty((T, self.n), dtype=td, device=self.device)
        _need(z, (T, self.n), td, self.device, "z")
        if save8 and self.fold:
            raise ValueError("save8: the layer folds its blocks into the weight (fold != 0)")
        if save and y is None:
            y = (self._new_checkpoint(T, self.n) if save8 else
                 torch.empty((T, self.n), dtype=td, device=self.device))
        if save and save_xg and xg is None:
            xg = (self._new_checkpoint(T, self.m) if save8 else
                  torch.empty((T, self.m), dtype=td, device=self.device))
        y = y if save else None
        xg = xg if save and save_xg else None
        for name, t, d in (("y", y, self.n), ("xg", xg, self.m)):
            if t is not None:
                self._need_saved(t, T, d, name, save8)
        with self._on(stream):
            self._dequantize(stream)
            L = self._abi()
            q8 = self._q8(y, xg)
            if q8 is None:
                nb = poetx_forward_workspace_bytes(L, T)
                ws = self.workspace("fwd", nb, stream)
                poetx_forward(L, T, x, z, y, xg, ws, nb, stream)
            else:
                nb = poetx_forward_q8_workspace_bytes(L, T, q8)
                ws = self.workspace("fwd", nb, stream)
                poetx_forward_q8(L, T, x, z, None if save8 else y, None if save8 else xg, q8, ws, nb, stream)
        return z, (Saved(y, xg) if save else None)

    def _need_saved(self, t, T: int, d: int, name: str, as_checkpoint: bool) -> None:
        if as_checkpoint != isinstance(t, Checkpoint):
            raise TypeError(f"{name}: expected a {'Checkpoint' if as_checkpoint else 'torch.Tensor'}, "
                            f"got {type(t).__name__}")
        if as_checkpoint:
            _need(t.codes, (T, d), torch.int8, self.device, f"{name} codes")
            _need(t.exps, (T, (d + 31) // 32), torch.uint8, self.device, f"{name} exps")
        else:
            _need(t, (T, d), self.torch_dtype, self.device, name)

    def backward(self, x: torch.Tensor, saved, dz: torch.Tensor, need_dx: bool = True,
                 dx: Optional[torch.Tensor] = None, dqR: Optional[torch.Tensor] = None,
                 dqP: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None):
        """dx, dqR, dqP of L = <dz, z>.  `saved` is what forward returned (or
        just the saved Y tensor); None recomputes Y from x (the "mem" variant,
        which keeps no [T][n] activation between forward and backward)."""
        if saved is None:
            saved = Saved(None, None)
        elif isinstance(saved, (torch.Tensor, Checkpoint)):
            saved = Saved(saved, None)
        T = dz.shape[0]
        if need_dx and dx is None:
            dx = torch.empty((T, self.m), dtype=self.torch_dtype, device=self.device)
        if dqR is None:
            dqR = torch.empty_like(self.qR)
        if dqP is None:
            dqP = torch.empty_like(self.qP)
        self._check_backward(T, x, saved, dz, dx if need_dx else None)
        _need(dqR, tuple(self.qR.shape), torch.float32, self.device, "dqR")
        _need(dqP, tuple(self.qP.shape), torch.float32, self.device, "dqP")
        self._backward(poetx_backward, poetx_backward_q8, T, x, saved, dz, dx if need_dx else None, dqR, dqP, accumulate,
                       stream)
        return (dx if need_dx else None), dqR, dqP

    def backward_dG(self, x: torch.Tensor, saved, dz: torch.Tensor, dGR: torch.Tensor, dGP: torch.Tensor,
                    need_dx: bool = True, dx: Optional[torch.Tensor] = None, accumulate: bool = False,
                    stream=None) -> Optional[torch.Tensor]:
        """backward() up to the token sums dGR [m/b][b][b], dGP [n/b][b][b]
        (fp32), without the CNP backward; LayerGroup.cnp_backward turns the dG
        of all layers into dq in one batch."""
        if saved is None:
            saved = Saved(None, None)
        elif isinstance(saved, (torch.Tensor, Checkpoint)):
            saved = Saved(saved, None)
        T = dz.shape[0]
        if need_dx and dx is None:
            dx = torch.empty((T, self.m), dtype=self.torch_dtype, device=self.device)
        self._check_backward(T, x, saved, dz, dx if need_dx else None)
        _need(dGR, (self.m // self.b, self.b, self.b), torch.float32, self.device, "dGR")
        _need(dGP, (self.n // self.b, self.b, self.b), torch.float32, self.device, "dGP")
        self._backward(poetx_backward_dG, poetx_backward_dG_q8, T, x, saved, dz, dx if need_dx else None, dGR, dGP,
                       accumulate, stream)
        return dx if need_dx else None

    def _backward(self, call, call_q8, T: int, x, saved: "Saved", dz, dx, gR, gP, accumulate: bool, stream) -> None:
        with self._on(stream):
            self._dequantize(stream)
            L = self._abi()
            q8 = self._q8(saved.y, saved.xg)
            y = None if isinstance(saved.y, Checkpoint) else saved.y
            xg = None if isinstance(saved.xg, Checkpoint) else saved.xg
            if q8 is None:
                nb = (poetx_backward_workspace_bytes if y is not None else
                      poetx_backward_recompute_workspace_bytes)(L, T)
                ws = self.workspace("bwd", nb, stream)
                call(L, T, x, y, xg, dz, dx, gR, gP, int(accumulate), ws, nb, stream)
            else:
                nb = poetx_backward_q8_workspace_bytes(L, T, int(y is not None), q8)
                ws = self.workspace("bwd", nb, stream)
                call_q8(L, T, x, y, xg, q8, dz, dx, gR, gP, int(accumulate), ws, nb, stream)

    def _check_backward(self, T: int, x, saved: "Saved", dz, dx) -> None:
        td = self.torch_dtype
        _need(dz, (T, self.n), td, self.device, "dz")
        if x is not None:
            _need(x, (T, self.m), td, self.device, "x")
        elif saved.xg is None:
            raise ValueError("x: needed unless the forward saved Xg")
        if self.fold and (isinstance(saved.y, Checkpoint) or isinstance(saved.xg, Checkpoint)):
            raise ValueError("saved: checkpoints, but the layer folds its blocks into the weight (fold != 0)")
        for name, t, d in (("saved y", saved.y, self.n), ("saved xg", saved.xg, self.m)):
            if t is not None:
                self._need_saved(t, T, d, name, isinstance(t, Checkpoint))
        if dx is not None:
            _need(dx, (T, self.m), td, self.device, "dx")

    def merge(self, new_permR: torch.Tensor, new_permP: torch.Tensor, stream=None) -> None:
        """W0 <- R W0 P, re-expressed in the frame of the new permutations;
        q = 0 and G = I afterwards.  The merged weight of a quantized layer is
        quantized again, into the same codes and scales."""
        self._need_weight("merge")
        with self._on(stream):
            self._dequantize(stream)
            L = self.abi()
            nb = poetx_merge_workspace_bytes(L)
            ws = self.workspace("merge", nb, stream)
            W_out = torch.empty_like(self.W)
            newR = new_permR.to(device=self.device, dtype=torch.int32).contiguous()
            newP = new_permP.to(device=self.device, dtype=torch.int32).contiguous()
            _need(newR, (self.m,), torch.int32, self.device, "new_permR")
            _need(newP, (self.n,), torch.int32, self.device, "new_permP")
            poetx_merge(L, newR, newP, W_out, ws, nb, stream)
            if self.Wq is None:
                _drop(self.W, stream)
                self.W = W_out
            else:
                poetx_weight_quantize(self.n, self.m, W_out, self.dtype, self.Wq, self.Wscale, stream)
            self.permR.copy_(newR)
            self.permP.copy_(newP)


class Int8Linear:
    """A linear z = x W^T served in 8 bits: the weight as int8 codes with a
    scale per row, tokens as int8 rows (rmsnorm_quantize or quantize_rows), the
    product in int8.  from_layer takes a trained POET-X layer with its R and P
    folded into the weight; the layer itself stays as it is."""

    def __init__(self, W: torch.Tensor, stream=None):
        if not isinstance(W, torch.Tensor) or W.dim() != 2 or W.dtype not in _TORCH_DTYPE.values():
            raise ValueError("W: expected a [n][m] torch.bfloat16 or torch.float32 tensor")
        if not W.is_contiguous():
            raise ValueError("W: must be contiguous")
        if W.device.type != "cuda":
            raise ValueError(f"W: tensor on {W.device}: the library runs on CUDA devices")
        self.n, self.m = W.shape
        self.dtype = W.dtype
        self.Wq = torch.empty((self.n, self.m), dtype=torch.int8, device=W.device)
        self.wscale = torch.empty(self.n, dtype=torch.float32, device=W.device)
        code = next(k for k, v in _TORCH_DTYPE.items() if v == W.dtype)
        with _on(stream, W.device):
            poetx_weight_quantize(self.n, self.m, W, code, self.Wq, self.wscale, stream)

    @classmethod
    def from_layer(cls, layer: PoetxLinear, stream=None) -> "Int8Linear":
        """The served form of a layer.  With `stream` the work runs there, after
        what the current stream holds and before what is queued on it later."""
        layer._need_weight("from_layer")
        here = torch.cuda.current_stream(layer.device)
        there = _torch_stream(stream, layer.device) or here
        if there != here:
            there.wait_stream(here)
        # every copy and temporary belongs to the stream that uses it
        with _on(there, layer.device):
            layer._dequantize(there)
            # merge a copy of the layer's state into the natural order (identity permutations)
            keep = [t.clone() for t in (layer.qR, layer.qP, layer.GR, layer.GP)]
            L = make_layer(layer.m, layer.n, layer.b, layer.dtype, layer.W, layer.permR, layer.permP, *keep)
            eyeR = torch.arange(layer.m, dtype=torch.int32, device=layer.device)
            eyeP = torch.arange(layer.n, dtype=torch.int32, device=layer.device)
            W = torch.empty((layer.n, layer.m), dtype=layer.torch_dtype, device=layer.device)
            nb = poetx_merge_workspace_bytes(L)
            ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=layer.device)
            poetx_merge(L, eyeR, eyeP, W, ws, nb, there)
            lin = cls(W, there)
        if there != here:
            here.wait_stream(there)
            for t in (lin.Wq, lin.wscale):
                t.record_stream(here)
        return lin

    def forward(self, x) -> torch.Tensor:
        """z [T][n] from tokens [T][m] (quantized here) or from their int8 rows
        (anything with .codes and .scale: QuantRows, NormRows)."""
        rows = quantize_rows(x) if isinstance(x, torch.Tensor) else x
        return matmul_int8(rows.codes, rows.scale, self.Wq, self.wscale, self.dtype)

    def backward(self, dz: torch.Tensor) -> torch.Tensor:
        """dx [T][m] of the tokens from dz [T][n], in 8 bits too."""
        return matmul_int8_grad(dz, self.Wq, self.wscale)


class LayerGroup:
    """Several layers with the same b and dtype whose G blocks are rebuilt
    together (one batched CNP build for all of them), optionally with their
    packed triangles in one flat buffer (qR then qP of each layer, in order)
    so one optimizer launch updates all of them."""

    def __init__(self, layers):
        self.layers = list(layers)
        self._ws = {}
        self.q = None
        self.m1 = None
        self.m2 = None
        self.steps = 0

    def flatten_params(self) -> torch.Tensor:
        """Move every layer's qR, qP into one flat fp32 buffer (the layers keep
        views into it) and allocate the optimizer moments; returns the buffer."""
        total = sum(L.qR.numel() + L.qP.numel() for L in self.layers)
        dev = self.layers[0].device
        self.q = torch.empty(total, dtype=torch.float32, device=dev)
        off = 0
        for L in self.layers:
            for name in ("qR", "qP"):
                t = getattr(L, name)
                view = self.q[off:off + t.numel()].view_as(t)
                view.copy_(t)
                setattr(L, name, view)
                off += t.numel()
        self.m1 = torch.zeros_like(self.q)
        self.m2 = torch.zeros_like(self.q)
        return self.q

    def optimizer_step(self, grad: torch.Tensor, lr: float, beta1: float = 0.9, beta2: float = 0.95,
                       eps: float = 1e-8, weight_decay: float = 0.0, stream=None) -> None:
        """AdamW on the flat packed triangles with the flat gradient `grad`
        (same layout), then the batched CNP rebuild of every G."""
        if self.q is None:
            raise RuntimeError("flatten_params() first")
        _need(grad, tuple(self.q.shape), torch.float32, self.q.device, "grad")
        self.steps += 1
        with _on(stream, self.q.device):
            poetx_adamw_step(self.q.numel(), self.q, grad, self.m1, self.m2, lr, beta1, beta2, eps, weight_decay,
                             self.steps, stream)
        self.build(stream)

    def dG_buffer(self) -> torch.Tensor:
        """A flat fp32 buffer [sum of blocks][b][b] for the dG of every layer,
        blocks in the order of the packed triangles (R then P of each layer)."""
        b = self.layers[0].b
        nblk = sum(L.m // b + L.n // b for L in self.layers)
        return torch.empty((nblk, b, b), dtype=torch.float32, device=self.layers[0].device)

    def dG_views(self, dG: torch.Tensor):
        """(dGR, dGP) views of each layer into a dG_buffer()."""
        out, off = [], 0
        for L in self.layers:
            nR, nP = L.m // L.b, L.n // L.b
            out.append((dG[off:off + nR], dG[off + nR:off + nR + nP]))
            off += nR + nP
        return out

    def cnp_backward(self, dG: torch.Tensor, dq: torch.Tensor, accumulate: bool = False, stream=None) -> None:
        """dq (flat, the layout of flatten_params) from the dG of every layer
        (dG_buffer layout): one batched CNP backward over all blocks."""
        if self.q is None:
            raise RuntimeError("flatten_params() first")
        L0 = self.layers[0]
        nblk = sum(L.m // L.b + L.n // L.b for L in self.layers)
        _need(dG, (nblk, L0.b, L0.b), torch.float32, self.q.device, "dG")
        _need(dq, tuple(self.q.shape), torch.float32, self.q.device, "dq")
        with _on(stream, self.q.device):
            nb = poetx_cnp_workspace_bytes(nblk, L0.b, L0.dtype)
            ws = _workspace(self._ws, "bwd", nb, L0.device, stream)
            poetx_cnp_backward(nblk, L0.b, self.q, dG, dq, int(accumulate), L0.dtype, ws, nb, stream)

    def build(self, stream=None) -> None:
        with self.layers[0]._on(stream):
            abis = [L._abi() for L in self.layers]
            nb = poetx_layers_cnp_workspace_bytes(abis)
            ws = _workspace(self._ws, "build", nb, self.layers[0].device, stream)
            poetx_layers_cnp_build(abis, ws, nb, stream)
