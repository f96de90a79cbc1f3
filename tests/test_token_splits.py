"""Token sums of bf16 layers whose products take the K-split GEMM (blocks other
than 256, and the P side with its block product folded into the weight): token
counts at which the 64-token steps do not fill every split, so that the last
ones would be left without a token.

Tolerance: fp32 accumulation on the tensor cores cuts off up to a whole step
2^-23 a term: 2 u24 of the sum of magnitudes for each of T terms and the splits."""
import pytest
import torch

import orthogonal_equivalence_b200 as px
from orthogonal_equivalence_b200 import build as pbuild

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U24 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pbuild.build()
    px.lib()
    px.poetx_device_error()
    yield
    torch.cuda.synchronize()
    assert px.poetx_device_error() == 0


def rnd(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def unused_splits(nblk, b, T):
    """How many of the splits that fill 148 SMs with tiles of 128 x (256, 128 or 64), four 64-token steps a split at
    least, get no step when each takes as many as the first."""
    tiles = nblk * -(-b // 128) * (b // (256 if b % 256 == 0 else 128 if b % 128 == 0 else 64))
    steps = -(-T // 64)
    s = max(1, min(148 // tiles, steps // 4, 32))
    return s - -(-steps // -(-steps // s))


# (d, b, T) whose last splits would be empty: 33 steps for 8 splits of 5, 37 and 55 for 9, 45 for 11, ...
EMPTY = [(192, 64, 2100), (1024, 64, 2340), (768, 64, 2850), (64, 64, 3500), (512, 128, 2700), (640, 128, 4400), (1024, 512, 2340),
         (512, 512, 4097)]


def dirty_tmem():
    """Leaves large numbers in the accumulators of every SM."""
    x = torch.full((1, 4096), 127, dtype=torch.int8, device="cuda")
    one = torch.full((1,), 1e30, device="cuda")
    for T in (2, 4096):
        px.matmul_int8(x.expand(T, -1).contiguous(), one.expand(T).contiguous(), x.expand(4096, -1).contiguous(),
                       one.expand(4096).contiguous())
    a = torch.full((4096, 1024), 3e18, dtype=BF, device="cuda")
    L = px.PoetxLinear(1024, 1024, 64, px.POETX_BF16)
    eye = torch.arange(1024, dtype=torch.int32, device="cuda")
    L.load(torch.full((1024, 1024), 3e18, dtype=BF, device="cuda"), eye, eye, torch.zeros_like(L.qR), torch.zeros_like(L.qP))
    L.forward(a)


def near(got, X, D, T, b):
    X, D = (v.double().view(T, -1, b) for v in (X, D))
    want, size = torch.einsum("tjr,tjc->jrc", X, D), torch.einsum("tjr,tjc->jrc", X.abs(), D.abs())
    return bool(((got.double() - want).abs() <= 2 * (T + 34) * U24 * size).all())


def test_the_cases_have_splits_without_tokens():
    assert all(unused_splits(d // b, b, T) > 0 for d, b, T in EMPTY)


@pytest.mark.parametrize("d,b,T", EMPTY)
def test_block_backward_from_a_checkpoint(d, b, T):
    D, G = rnd(1, T, d, dtype=BF), rnd(2, d // b, b, b, dtype=BF)
    c = px.checkpoint_save(rnd(3, T, d, dtype=BF))
    for _ in range(2):
        dirty_tmem()
        _, dG = px.block_backward(c, D, G, need_o=False)
        assert near(dG, px.checkpoint_load(c, F32), D, T, b)


@pytest.mark.parametrize("fold,b,T", [(0, b, T) for _, b, T in EMPTY] +
                         [(px.POETX_FOLD_P, 256, 4672), (px.POETX_FOLD_P, 256, 2340), (px.POETX_FOLD_P, 64, 2340)])
@pytest.mark.parametrize("save8", [False, True])
def test_a_layers_backward(fold, b, T, save8):
    if fold and save8:
        pytest.skip("a folding layer keeps no checkpoints")
    d = {t[1:]: t[0] for t in EMPTY}.get((b, T), 1024)
    m = n = d
    L = px.PoetxLinear(m, n, b, px.POETX_BF16, fold=fold)
    g = torch.Generator().manual_seed(4)
    L.load(rnd(5, n, m, dtype=BF, scale=0.05), torch.randperm(m, generator=g).int().cuda(),
           torch.randperm(n, generator=g).int().cuda(), torch.zeros_like(L.qR), torch.zeros_like(L.qP))     # G = I
    x, dz = rnd(6, T, m, dtype=BF), rnd(7, T, n, dtype=BF)
    _, saved = L.forward(x, save_xg=True, save8=save8)
    y, xg = ((px.checkpoint_load(c, F32) for c in saved) if save8 else saved)
    for need_dx in (True, False):
        dGR, dGP = torch.empty(m // b, b, b, device="cuda"), torch.empty(n // b, b, b, device="cuda")
        dirty_tmem()
        dx = L.backward_dG(None, saved, dz, dGR, dGP, need_dx=need_dx)
        if need_dx:
            dU = dx[:, L.permR.long()]      # (G = I: what the R side's sum multiplies)
        assert near(dGP, y, dz[:, L.permP.long()], T, b), "dGP"
        assert near(dGR, xg, dU, T, b), "dGR"
        dirty_tmem()
        a = L.backward(None, saved, dz, need_dx=need_dx)
        # at q = 0 the Cayley-Neumann map's derivative is 2 dQ: dq = 2 (dG - dG^T)
        i, j = torch.triu_indices(b, b, 1)
        for dq, dG in zip(a[1:], (dGR, dGP)):
            want = 2 * (dG - dG.transpose(1, 2))[:, i, j]
            assert (dq - want).abs().max() <= 2e-2 * dG.abs().max(), "dq"
