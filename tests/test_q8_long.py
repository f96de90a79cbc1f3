"""The 8-bit operators over many rows: sums over long ranges of tokens, and
blocks of threads that take several rows or tiles in turn.

u24 = 2^-24 is half a step of fp32.  The tensor core adds the 16 tokens of an
instruction to its fp32 sum at a time and cuts off what the addition shifts
out: the terms' and the sum's own step, two whole steps 2^-23 of the sum so far
at most."""
import pytest
import torch

import orthogonal_equivalence_b200 as px
from orthogonal_equivalence_b200 import build as pbuild

BF, F32 = torch.bfloat16, torch.float32
U24 = 2.0 ** -24
SPLIT = 2048 + 256      # most tokens of one sum: about 2048, to whole tiles


@pytest.fixture(scope="module")
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pbuild.build()
    px.lib()
    px.poetx_device_error()
    yield
    torch.cuda.synchronize()
    assert px.poetx_device_error() == 0


def rnd(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# ---------------------------------------------------------------- token sums
@pytest.mark.parametrize("T", [2049, 16384, 70001])
@pytest.mark.parametrize("b", [64, 128, 256, 512])
def test_partial_sums_for_every_2048_tokens(b, T):
    pbuild.build()
    d = 8192
    expanded = 0 if b == 256 else 2 * T * d     # X in bf16, where no kernel reads the codes
    sums = -(-T // 2048) * 4 * d * b
    assert px.poetx_block_backward_workspace_bytes(T, d, b, px.POETX_BF16) >= expanded + sums
    # the layer's backward from checkpoints sums the same way
    L = px.poetx_layer(d, d, b, px.POETX_BF16, 16, 16, 16, 16, 16, 16, 16, 0)
    kept = px.poetx_q8(None, None, 16, 16, 16, 16)
    more = px.poetx_backward_q8_workspace_bytes(L, T, 0, kept) - px.poetx_backward_q8_workspace_bytes(L, T, 1, px.poetx_q8())
    assert more >= expanded + 2 * sums


@pytest.mark.parametrize("dtype", [px.POETX_BF16, px.POETX_FP32])
@pytest.mark.parametrize("b", [64, 128, 256, 512])
def test_sizes_of_few_tokens(b, dtype):
    pbuild.build()
    L = px.poetx_layer(1024, 512, b, dtype, 16, 16, 16, 16, 16, 16, 16, 0)
    for T in (0, 1, 63, 64, 65, 129):
        assert px.poetx_block_backward_workspace_bytes(T, 1024, b, dtype) >= 4 * 1024 * b
        for q in (px.poetx_q8(), px.poetx_q8(16, 16, 16, 16, 16, 16)):
            assert px.poetx_backward_q8_workspace_bytes(L, T, 0, q) >= 4 * (1024 + 512) * b


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(16384, 8192), (5000, 8192), (16384, 1024)])
@pytest.mark.parametrize("b", [64, 128, 256, 512])
def test_long_token_sums(gpu, b, T, d):
    # terms of one sign: what an addition cuts off adds up.  A sum of S tokens is S / 16 additions to a sum that
    # grows evenly, half of the last on average, so it loses (S / 16 + 1) 2^-23 of itself at most; then the splits'
    # sums are added, each addition rounded.
    x, D = rnd(1, T, d, dtype=BF).abs(), rnd(2, T, d, dtype=BF).abs()
    c = px.checkpoint_save(x)
    _, dG = px.block_backward(c, D, rnd(3, d // b, b, b, dtype=BF), need_o=False)
    X = px.checkpoint_load(c, F32)
    bound = (SPLIT / 16 + 1) * 2 * U24 + (-(-T // 1024) + 1) * U24
    for j in range(0, d // b, max(1, d // b // 8)):
        want = X[:, j * b:(j + 1) * b].double().t() @ D[:, j * b:(j + 1) * b].double()
        assert ((dG[j].double() - want).abs() <= bound * want).all()


# ---------------------------------------------------------------- the longest rows
@pytest.mark.gpu
@pytest.mark.parametrize("d", [2 ** 31 - 16, 2 ** 31 - 1])
def test_a_row_as_long_as_an_int(gpu, d):
    codes = torch.arange(-128, 128, device="cuda").to(torch.int8).repeat(d // 256 + 1)[:d].view(1, d)
    scale = torch.tensor([0.37], device="cuda")
    w = px.dequantize_rows(codes, scale, BF)
    one = (torch.arange(-128, 128, device="cuda").float() * scale).to(BF)
    assert torch.equal(w[0, :d // 256 * 256].view(-1, 256), one.expand(d // 256, 256))
    assert torch.equal(w[0, d // 256 * 256:], one[:d % 256])


# ---------------------------------------------------------------- several rows or tiles in turn
# More rows than the grid has blocks (at most 16 blocks a SM), so that a block loads its next row while it
# works on one and keeps its share of dgamma over all of them: every register shape of the row kernels, with
# whole rows and cut ones, bf16 and fp32.
TURNS = [(3000, 512), (2500, 1024), (3000, 2048), (1500, 4096), (1300, 3584), (900, 5120), (1200, 7168), (700, 8192),
         (700, 14336), (500, 16384), (5001, 264), (2600, 648)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", TURNS)
def test_blocks_that_take_several_rows(gpu, T, d, dtype):
    from test_q8_gpu import test_quantize_rows, test_rmsnorm_backward, test_rmsnorm_quantize
    test_quantize_rows(T, d, dtype)
    for residual in (False, True):
        test_rmsnorm_quantize(T, d, residual, dtype)
        test_rmsnorm_backward(T, d, residual, dtype)


# More items (block, token split) than the 74 pairs of SMs, with values everywhere: a pair's second item takes over
# the accumulators, the resident G and every ring in mid-phase; and other blocks beside them.
@pytest.mark.gpu
@pytest.mark.parametrize("T,d,b", [(16384, 2304, 256), (5000, 8192, 256), (300, 38400, 256), (1, 25600, 256), (16384, 4096, 256),
                                   (12345, 5120, 512), (9000, 1920, 64), (7001, 2688, 128)])
def test_blocks_of_more_items_than_pairs(gpu, T, d, b):
    D, G = rnd(11, T, d, dtype=BF), rnd(12, d // b, b, b, dtype=BF, scale=0.3)
    c = px.checkpoint_save(rnd(10, T, d, dtype=BF))
    O, dG = px.block_backward(c, D, G)
    none, alone = px.block_backward(c, D, G, need_o=False)
    assert none is None and torch.equal(alone, dG)
    X = px.checkpoint_load(c, F32)
    terms = min(T, SPLIT) + -(-T // 1024) + 34      # of a sum: a split's tokens, then the splits
    for j in range(d // b):
        at = slice(j * b, (j + 1) * b)
        Dj, Gj, Xj = D[:, at].double(), G[j].double(), X[:, at].double()
        want, size = Dj @ Gj.t(), Dj.abs() @ Gj.abs().t()
        # fp32 accumulation, up to a whole step cut off a term; O is rounded to bf16
        assert ((O[:, at].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * (b + 2) * U24 * size).all(), ("O", j)
        want, size = Xj.t() @ Dj, Xj.abs().t() @ Dj.abs()
        assert ((dG[j].double() - want).abs() <= 2 * terms * U24 * size).all(), ("dG", j)


# Tiles of 128 tokens by the weight's rows: one wave of them for up to 128 tokens of a wide weight, and a long K
# split in two; and many tiles on each pair.
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,m,n", [(100, 256, 20000), (128, 512, 19201), (512, 8192, 4096), (500, 9000, 4000),
                                   (3000, 384, 6000), (9001, 128, 4096)])
def test_wide_and_many_int8_tiles(gpu, T, m, n, dtype):
    from test_q8_gpu import test_matmul_int8, test_matmul_int8_grad
    test_matmul_int8(T, m, n, dtype)
    test_matmul_int8_grad(T, n, m, dtype)      # the same tiles, the weight's rows as K
    test_matmul_int8_grad(T, m, n, dtype)
