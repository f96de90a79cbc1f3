"""The C calls of the 8-bit path through their ctypes wrappers, with buffers of
the caller's own: the results of the torch functions, which call the same
library."""
import pytest
import torch

import orthogonal_equivalence_b200 as px
from orthogonal_equivalence_b200 import build as pbuild

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DT = {BF: px.POETX_BF16, F32: px.POETX_FP32}


@pytest.fixture(scope="module", autouse=True)
def library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pbuild.build()
    px.lib()


def rnd(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def scratch(nbytes):
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda"), nbytes


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d,n,b", [(37, 192, 80, 64), (300, 1024, 513, 256)])
def test_the_wrappers_give_the_functions_results(T, d, n, b, dtype):
    pd = DT[dtype]
    x, r, gamma = rnd(1, T, d, dtype=dtype), rnd(2, T, d, dtype=dtype), rnd(3, d) + 1
    q, s = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    px.poetx_quantize_rows(T, d, x, pd, gamma, q, s)
    for a, w in zip((q, s), px.quantize_rows(x, gamma)):
        assert torch.equal(a, w)
    want = px.rmsnorm_quantize(x, gamma, r, 1e-5, y=True)
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty_like(s)
    px.poetx_rmsnorm_quantize(T, d, x, r, gamma, 1e-5, pd, h, y, q, s, rstd)
    for a, w in zip((q, s, h, rstd, y), want):
        assert torch.equal(a, w)
    dx, dgamma = torch.empty_like(x), torch.empty_like(gamma)
    px.poetx_rmsnorm_backward(T, d, x, h, gamma, rstd, r, pd, dx, dgamma, 0,
                              *scratch(px.poetx_rmsnorm_backward_workspace_bytes(T, d, pd)))
    for a, w in zip((dx, dgamma), px.rmsnorm_backward(x, h, gamma, rstd, r)):
        assert torch.equal(a, w)
    W = px.quantize_rows(rnd(4, n, d))
    z = torch.empty(T, n, dtype=dtype, device="cuda")
    px.poetx_matmul_int8(T, n, d, q, s, W.codes, W.scale, pd, z, *scratch(px.poetx_matmul_int8_workspace_bytes(T, n, d)))
    assert torch.equal(z, px.matmul_int8(q, s, *W, dtype))
    px.poetx_matmul_int8_grad(T, n, d, z, W.codes, W.scale, pd, dx,
                              *scratch(px.poetx_matmul_int8_grad_workspace_bytes(T, n, d)))
    assert torch.equal(dx, px.matmul_int8_grad(z, *W))
    c, e = torch.empty_like(q), torch.empty(T, (d + 31) // 32, dtype=torch.uint8, device="cuda")
    px.poetx_checkpoint_save(T, d, x, pd, c, e)
    kept = px.checkpoint_save(x)
    assert torch.equal(c, kept.codes) and torch.equal(e, kept.exps)
    px.poetx_checkpoint_load(T, d, c, e, pd, y)
    assert torch.equal(y, px.checkpoint_load(kept, dtype))
    G, O, dG = rnd(5, d // b, b, b, dtype=dtype), torch.empty_like(x), torch.empty(d // b, b, b, device="cuda")
    px.poetx_block_backward(T, d, b, c, e, r, G, pd, O, dG, 0,
                            *scratch(px.poetx_block_backward_workspace_bytes(T, d, b, pd)))
    for a, w in zip((O, dG), px.block_backward(kept, r, G)):
        assert torch.equal(a, w)
