"""The 8-bit operators refuse what they cannot take before anything is queued:
the C calls by status, the torch functions by exception (no GPU needed)."""
import ctypes

import pytest
import torch

import orthogonal_equivalence_b200 as px
from orthogonal_equivalence_b200 import build as pbuild

BF = torch.bfloat16
P, ODD, WS = 4096, 4100, 1 << 40   # aligned and unaligned addresses, a large workspace


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return px.lib()


def test_statuses_of_the_rows(lib):
    q = lib.poetx_quantize_rows
    assert q(4, 64, P, 7, None, P, P, None) == 3
    assert q(-1, 64, P, 1, None, P, P, None) == 1
    assert q(4, 0, P, 1, None, P, P, None) == 1
    assert q(4, 102401, P, 1, None, P, P, None) == 2
    assert q(2 ** 31, 64, P, 1, None, P, P, None) == 2
    assert q(4, 64, None, 1, None, P, P, None) == 1
    assert q(4, 64, P, 1, ODD, P, P, None) == 4
    assert q(4, 64, P, 1, None, ODD, P, None) == 4
    assert q(0, 64, None, 1, None, None, None, None) == 0


def test_statuses_of_the_norm(lib):
    n = lib.poetx_rmsnorm_quantize
    assert n(4, 64, P, None, P, 1e-5, 5, None, None, P, P, None, None) == 3
    assert n(4, 51201, P, None, P, 1e-5, 1, None, None, P, P, None, None) == 2
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert n(4, 64, P, None, P, eps, 1, None, None, P, P, None, None) == 1
    assert n(4, 64, P, None, P, 1e-5, 1, None, None, None, None, P, None) == 1    # nothing asked for
    assert n(4, 64, P, None, P, 1e-5, 1, None, None, P, None, P, None) == 1       # codes without scales
    assert n(4, 64, P, P, P, 1e-5, 1, None, None, P, P, P, None) == 1             # residual without h
    assert n(4, 64, P, None, None, 1e-5, 1, None, None, P, P, P, None) == 1
    assert n(4, 64, P, None, P, 1e-5, 1, None, ODD, P, P, P, None) == 4
    b = lib.poetx_rmsnorm_backward
    need = px.poetx_rmsnorm_backward_workspace_bytes(4, 64, 1)
    assert need > 0 and px.poetx_rmsnorm_backward_workspace_bytes(4, 51201, 1) == 0
    assert b(4, 64, P, P, P, P, None, 1, P, P, 0, P, need - 1, None) == 5
    assert b(4, 64, P, P, P, P, None, 1, P, P, 0, None, need, None) == 5
    assert b(4, 64, P, P, P, None, None, 1, P, P, 0, P, need, None) == 1
    assert b(4, 64, P, P, P, P, ODD, 1, P, P, 0, P, need, None) == 4
    assert b(4, 64, P, P, P, P, None, 1, P, None, 0, P, need, None) == 1


def test_statuses_of_the_products(lib):
    f = lib.poetx_matmul_int8
    assert f(4, 64, 64, P, P, P, P, 3, P, None, 0, None) == 3
    assert f(4, 102401, 64, P, P, P, P, 1, P, None, 0, None) == 2
    assert f(4, 64, 102401, P, P, P, P, 1, P, None, 0, None) == 2
    assert f(4, 64, 0, P, P, P, P, 1, P, None, 0, None) == 1
    assert f(4, 64, 64, P, None, P, P, 1, P, None, 0, None) == 1
    assert f(4, 64, 64, P, P, ODD, P, 1, P, None, 0, None) == 4
    need = px.poetx_matmul_int8_workspace_bytes(4, 64, 65)
    assert need > 0 and px.poetx_matmul_int8_workspace_bytes(4, 64, 64) == 0
    assert f(4, 64, 65, P, P, P, P, 1, P, P, need - 1, None) == 5
    assert f(4, 64, 65, P, P, P, P, 1, P, None, need, None) == 5
    g = lib.poetx_matmul_int8_grad
    need = px.poetx_matmul_int8_grad_workspace_bytes(4, 64, 64)
    assert need > 0 and px.poetx_matmul_int8_grad_workspace_bytes(4, 0, 64) == 0
    assert g(4, 64, 64, P, P, P, 1, P, P, need - 1, None) == 5
    assert g(4, 64, 64, P, P, None, 1, P, P, need, None) == 1
    assert g(-4, 64, 64, P, P, P, 1, P, P, need, None) == 1


def test_statuses_of_the_checkpoints(lib):
    s, l, b = lib.poetx_checkpoint_save, lib.poetx_checkpoint_load, lib.poetx_block_backward
    assert s(4, 64, P, 9, P, P, None) == 3
    assert s(4, 64, P, 1, P, None, None) == 1
    assert s(4, 64, P, 1, ODD, P, None) == 4
    assert l(4, 102401, P, P, 1, P, None) == 2
    need = px.poetx_block_backward_workspace_bytes(4, 128, 64, 1)
    assert need > 0 and px.poetx_block_backward_workspace_bytes(4, 128, 48, 1) == 0
    assert b(4, 128, 48, P, P, P, P, 1, P, P, 0, P, need, None) == 2    # bf16 wants b % 64 == 0
    assert b(4, 100, 64, P, P, P, P, 1, P, P, 0, P, need, None) == 2    # b divides d
    assert b(4, 128, 64, P, P, P, None, 1, P, P, 0, P, need, None) == 1  # O without G
    assert b(4, 128, 64, P, P, P, P, 1, P, ODD, 0, P, need, None) == 4
    assert b(4, 128, 64, P, P, P, P, 1, P, P, 0, P, need - 1, None) == 5


def test_torch_functions_refuse():
    x, q = torch.zeros(4, 64, dtype=BF), torch.zeros(4, 64, dtype=torch.int8)
    g, s = torch.ones(64), torch.ones(4)
    with pytest.raises(TypeError, match="x: expected"):
        px.quantize_rows([1.0])
    with pytest.raises(ValueError, match="x: dtype"):
        px.quantize_rows(x.half())
    with pytest.raises(ValueError, match="x: shape"):
        px.quantize_rows(x[0])
    with pytest.raises(ValueError, match="x: must be contiguous"):
        px.quantize_rows(torch.zeros(64, 4, dtype=BF).t())
    with pytest.raises(ValueError, match="colscale: shape"):
        px.quantize_rows(x, torch.ones(63))
    with pytest.raises(ValueError, match="CUDA"):
        px.quantize_rows(x)
    with pytest.raises(ValueError, match="gamma: dtype"):
        px.rmsnorm_quantize(x, g.to(BF))
    with pytest.raises(ValueError, match="residual: shape"):
        px.rmsnorm_quantize(x, g, x[:3])
    with pytest.raises(ValueError, match="rstd: shape"):
        px.rmsnorm_backward(x, x, g, g)
    with pytest.raises(ValueError, match="h: dtype"):
        px.rmsnorm_backward(x, x.float(), g, s)
    with pytest.raises(ValueError, match="Wq: shape"):
        px.matmul_int8(q, s, torch.zeros(8, 63, dtype=torch.int8), torch.ones(8))
    with pytest.raises(ValueError, match="xscale: shape"):
        px.matmul_int8(q, g, torch.zeros(8, 64, dtype=torch.int8), torch.ones(8))
    with pytest.raises(ValueError, match="dtype"):
        px.matmul_int8(q, s, torch.zeros(8, 64, dtype=torch.int8), torch.ones(8), torch.float16)
    with pytest.raises(ValueError, match="wscale: shape"):
        px.matmul_int8_grad(x, torch.zeros(64, 8, dtype=torch.int8), torch.ones(8))
    with pytest.raises(ValueError, match="checkpoint exps: shape"):
        px.checkpoint_load(px.Checkpoint(q, torch.zeros(4, 3, dtype=torch.uint8)), BF)
    ck = px.Checkpoint(q, torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="D: shape"):
        px.block_backward(ck, torch.zeros(3, 64, dtype=BF), torch.zeros(1, 64, 64, dtype=BF))
    with pytest.raises(ValueError, match="G: shape"):
        px.block_backward(ck, x, torch.zeros(1, 64, 32, dtype=BF))
    with pytest.raises(ValueError, match="G: dtype"):
        px.block_backward(ck, x, torch.zeros(1, 64, 64))


def test_statuses_of_the_layer_in_8_bits(lib):
    L = px.poetx_layer(512, 256, 64, px.POETX_BF16, P, P, P, P, P, P, P, 0)
    folded = px.poetx_layer(512, 256, 64, px.POETX_BF16, P, P, P, P, P, P, P, 1)
    q = px.poetx_q8(P, P, P, P, P, P)
    need = px.poetx_forward_q8_workspace_bytes(L, 10, q)
    assert need > px.poetx_forward_workspace_bytes(L, 10)
    assert px.poetx_backward_q8_workspace_bytes(L, 10, 0, q) > px.poetx_backward_workspace_bytes(L, 10)
    assert px.poetx_forward_q8_workspace_bytes(folded, 10, q) == 0
    f = lambda l, z, y, xg, q8, ws: lib.poetx_forward_q8(ctypes.byref(l), 10, P, z, y, xg, ctypes.byref(q8), P, ws, None)  # noqa: E731
    assert f(folded, P, None, None, q, need) == 1
    assert f(L, P, P, None, q, need) == 1                                   # Y in both forms
    assert f(L, P, None, P, q, need) == 1
    assert f(L, P, None, None, q, need - 1) == 5
    assert f(L, P, None, None, px.poetx_q8(P, None, None, None, None, None), need) == 1   # codes without scales
    assert f(L, P, None, None, px.poetx_q8(None, None, P, None, None, None), need) == 1
    assert f(L, P, None, None, px.poetx_q8(None, None, ODD, P, None, None), need) == 4
    assert lib.poetx_forward_q8(ctypes.byref(L), 10, P, P, None, None, None, P, need, None) == 1
    nb = px.poetx_backward_q8_workspace_bytes(L, 10, 0, q)
    b = lib.poetx_backward_q8
    assert b(ctypes.byref(L), 10, P, P, None, ctypes.byref(q), P, None, P, P, 0, P, nb, None) == 1
    assert b(ctypes.byref(L), 10, P, None, None, ctypes.byref(q), P, None, P, P, 0, P, nb - 1, None) == 5
    assert b(ctypes.byref(L), 10, P, None, None, ctypes.byref(q), None, None, P, P, 0, P, nb, None) == 1
    assert lib.poetx_backward_dG_q8(ctypes.byref(L), 10, P, None, None, ctypes.byref(q), P, None, None, P, 0, P, nb,
                                    None) == 1
