"""The 8-bit operators against plain 64-bit implementations on the same inputs.

Tolerances are worked out from the arithmetic, u24 = 2^-24 being half a step of
fp32 and half a step of bf16 2^-8: int8 codes, checkpoint values and the
rounded residual are exact; a value computed in fp32 by a chain of k roundings
is off by at most k u24 of the sum of the magnitudes that went into it; a bf16
result adds its own half step."""
import numpy as np
import pytest
import torch

import orthogonal_equivalence_b200 as px
from orthogonal_equivalence_b200 import build as pbuild

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U24}
BF, F32 = torch.bfloat16, torch.float32


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


def codes(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8).cuda()


def within(got, want, tol, what):
    """|got - want| <= tol elementwise (all in fp64), NaN where NaN is wanted."""
    got = got.double()
    assert got.shape == want.shape, what
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    off = ((got - want).abs() - tol).masked_fill(nan, 0.0)
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0, f"{what}: {int((off > 0).sum())} values outside, worst by {worst:.3e}"


def quantise64(u):
    """Codes (fp64) and scales (fp32) of fp32 rows, from the definition."""
    top = u.abs().max(1).values
    s = top / torch.full_like(top, 127.0)
    s = torch.where(torch.isfinite(u).all(1), s, torch.full_like(s, float("nan")))
    live = s > 0
    q = (u.double() / torch.where(live, s, torch.ones_like(s)).double()[:, None]).round().clamp(-127, 127)
    return torch.where(live[:, None], q, torch.zeros_like(q)), s


# ---------------------------------------------------------------- rows to int8
ROWS = [(1, 1), (1, 4096), (11, 9001), (3, 7), (5, 64), (77, 1000), (300, 1001), (130, 4096), (33, 5120), (9, 8200), (7, 14336),
        (5, 16383), (3, 20000), (2, 40001), (2, 102400)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", ROWS)
def test_quantize_rows(T, d, dtype):
    x = rnd(1, T, d, dtype=dtype)
    q, s = px.quantize_rows(x)
    qo, so = quantise64(x.float())
    assert torch.equal(s, so) and torch.equal(q.double(), qo)
    c = rnd(2, d).abs() + 0.1
    q, s = px.quantize_rows(x, c)
    qo, so = quantise64(x.float() * c)
    assert torch.equal(s, so) and torch.equal(q.double(), qo)


def test_quantize_rows_borders():
    # every value k / 2 of a row whose scale is exactly 1: all halves are ties, and go to the even code
    x = (torch.arange(-254, 255, dtype=F32) / 2).repeat(3, 1).cuda()
    x[1] *= 2.0 ** -120   # the same row near the bottom of the range
    x[2] *= 2.0 ** -145   # and as subnormals: the scale itself loses digits there
    q, s = px.quantize_rows(x)
    qo, so = quantise64(x)
    assert torch.equal(s, so) and torch.equal(q.double(), qo)
    assert s[0].item() == 1.0 and q[0, 1].item() == -126 and q[0, 3].item() == -126


@pytest.mark.parametrize("d", [40, 1001, 4096, 30000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_rows_zero_and_nonfinite(d, dtype):
    x = rnd(3, 5, d, dtype=dtype)
    x[0] = 0
    x[1, d // 2] = float("inf")
    x[2, d - 1] = float("nan")
    x[3, 0] = -float("inf")
    q, s = px.quantize_rows(x)
    assert s[0].item() == 0 and torch.isnan(s[1:4]).all() and not q[:4].any()
    qo, so = quantise64(x.float())
    assert torch.equal(q[4].double(), qo[4]) and s[4] == so[4]
    back = px.dequantize_rows(q, s, dtype)
    assert torch.isnan(back[1:4]).all() and not back[0].any()


# ---------------------------------------------------------------- norm
NORM = [(1, 1), (1, 4096), (11, 9001), (3, 7), (5, 64), (77, 1000), (300, 1001), (130, 4096), (33, 5120), (9, 8200), (7, 14336),
        (5, 16383), (3, 20000), (2, 40001), (2, 51200)]
EPS = 1e-5


def chain(d):
    """Roundings of a row's fp32 sum: a thread's own terms, then the tree of the block."""
    return max(32, d // 256 + 1) + 16


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,d", NORM)
def test_rmsnorm_quantize(T, d, residual, dtype):
    x, gamma = rnd(4, T, d, dtype=dtype), rnd(5, d) + 1
    r = rnd(6, T, d, dtype=dtype, scale=3) if residual else None
    n = px.rmsnorm_quantize(x, gamma, r, EPS, codes=True, y=True)
    h = (x.float() + r.float()).to(dtype) if residual else x
    assert torch.equal(n.h, h)
    rstd = (h.double().square().mean(1) + EPS).rsqrt()
    k = chain(d)
    within(n.rstd, rstd, k * U24 * rstd, "rstd")
    u = h.float() * gamma
    q, s = quantise64(u)
    assert torch.equal(n.codes.double(), q)
    within(n.scale, s.double() * rstd, (k + 1) * U24 * s.double() * rstd, "scale")
    y = u.double() * rstd[:, None]
    within(n.y, y, (HALF[dtype] * (1 + k * U24) + (k + 1) * U24) * y.abs(), "y")
    only = px.rmsnorm_quantize(x, gamma, r, EPS, codes=False, y=True)
    assert only.codes is None and torch.equal(only.y, n.y)


def test_rmsnorm_special_rows():
    x = rnd(7, 4, 512, dtype=BF)
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    gamma = rnd(8, 512)
    n = px.rmsnorm_quantize(x, gamma, None, EPS, y=True)
    assert n.scale[0] == 0 and not n.codes[0].any() and not n.y[0].any()
    assert torch.isnan(n.scale[1:3]).all() and not n.codes[1:3].any()
    assert torch.isnan(n.y[2]).all() and torch.isnan(n.y[1, 3])
    assert torch.isfinite(n.scale[3])


@pytest.mark.parametrize("d", [96, 1001, 4096, 20000])
def test_rmsnorm_in_place(d):
    # h over x or over the residual, y over x without a residual: the same results
    T = 5
    x, r, gamma = rnd(9, T, d, dtype=BF), rnd(10, T, d, dtype=BF), rnd(11, d)
    want = px.rmsnorm_quantize(x, gamma, r, EPS, y=True)
    for over in ("x", "r"):
        a, b = x.clone(), r.clone()
        h = a if over == "x" else b
        q, s, y = torch.empty_like(want.codes), torch.empty_like(want.scale), torch.empty_like(x)
        px.poetx_rmsnorm_quantize(T, d, a, b, gamma, EPS, px.POETX_BF16, h, y, q, s, None)
        assert torch.equal(h, want.h) and torch.equal(q, want.codes) and torch.equal(s, want.scale)
        assert torch.equal(y, want.y)
    a = x.clone()
    px.poetx_rmsnorm_quantize(T, d, a, None, gamma, EPS, px.POETX_BF16, None, a, None, None, None)
    assert torch.equal(a, px.rmsnorm_quantize(x, gamma, None, EPS, codes=False, y=True).y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,d", NORM + [(1500, 256), (700, 1000), (400, 999)])
def test_rmsnorm_backward(T, d, residual, dtype):
    dy, h, gamma = rnd(12, T, d, dtype=dtype), rnd(13, T, d, dtype=dtype), rnd(14, d) + 1
    dres = rnd(15, T, d, dtype=dtype) if residual else None
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dx, dg = px.rmsnorm_backward(dy, h, gamma, rstd, dres)
    rs, p = rstd.double()[:, None], dy.double() * gamma.double()
    xn = h.double() * rs
    mean = (p * xn).mean(1, keepdim=True)
    want = rs * (p - xn * mean)
    size = rs * (p.abs() + xn.abs() * (p * xn).abs().mean(1, keepdim=True))
    if residual:
        want = want + dres.double()
        size = size + dres.double().abs()
    k = chain(d) + 8
    within(dx, want, HALF[dtype] * want.abs() + 2 * k * U24 * size, "dx")
    terms = dy.double() * xn
    kt = -(-T // 148) + 160  # rows a block walks, then the partial sums
    within(dg, terms.sum(0), (kt + 3) * U24 * terms.abs().sum(0), "dgamma")
    # accumulation adds to what is there, and the call gives the same bits again
    acc = torch.ones_like(dg)
    dx2, out = px.rmsnorm_backward(dy, h, gamma, rstd, dres, dgamma=acc)
    assert out is acc and torch.equal(dx2, dx) and torch.equal(acc, 1 + dg)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", [(2500, 641), (1300, 1025), (900, 2261), (700, 4100), (400, 7169), (330, 14335), (310, 20001),
                                 (5, 24577)])
def test_rows_off_the_16_byte_units(T, d, dtype):
    # rows of any start within a unit, several to a block, with and without a gain; rows
    # of codes like the values' and on boundaries of their own (the gradient's)
    x, r, gamma = rnd(50, T, d, dtype=dtype), rnd(51, T, d, dtype=dtype), rnd(52, d) + 1
    q, s = px.quantize_rows(x)
    qo, so = quantise64(x.float())
    assert torch.equal(s, so) and torch.equal(q.double(), qo)
    n = px.rmsnorm_quantize(x, gamma, r, EPS, y=True)
    h = (x.float() + r.float()).to(dtype)
    assert torch.equal(n.h, h) and torch.equal(n.codes.double(), quantise64(h.float() * gamma)[0])
    y = (h.float() * gamma).double() * (h.double().square().mean(1, keepdim=True) + EPS).rsqrt()
    k = chain(d)
    within(n.y, y, (HALF[dtype] * (1 + k * U24) + (k + 1) * U24) * y.abs(), "y")
    W = rnd(53, d, 48, scale=40).round().clamp(-127, 127).to(torch.int8)
    qo, so = quantise64(x.float() * gamma)
    want = (qo @ W.double()) * so.double()[:, None]
    # the integer sum as fp32, times the scale, to the result's type
    within(px.matmul_int8_grad(x, W, gamma), want, (HALF[dtype] + 2.01 * U24) * want.abs(), "dx")
    test_rmsnorm_backward(T, d, True, dtype)


def test_rmsnorm_gradient_by_differences():
    # the same loss in 64 bits, moved by +-e along one direction of x and of gamma
    T, d = 6, 48
    x, gamma, dy = rnd(16, T, d), rnd(17, d) + 1, rnd(18, T, d)
    n = px.rmsnorm_quantize(x, gamma, None, EPS, y=True)
    dx, dg = px.rmsnorm_backward(dy, x, gamma, n.rstd)

    def loss(x_, g_):
        return (dy.double() * (x_ * (x_.square().mean(1, keepdim=True) + EPS).rsqrt() * g_)).sum().item()

    vx, vg, e = rnd(19, T, d).double(), rnd(20, d).double(), 1e-5
    x64, g64 = x.double(), gamma.double()
    num_x = (loss(x64 + e * vx, g64) - loss(x64 - e * vx, g64)) / (2 * e)
    num_g = (loss(x64, g64 + e * vg) - loss(x64, g64 - e * vg)) / (2 * e)
    # e^2 times a third derivative of order 1 per element, and fp32 sums of T*d terms of order 10
    assert abs(num_x - (dx.double() * vx).sum().item()) < 1e-3
    assert abs(num_g - (dg.double() * vg).sum().item()) < 1e-3


# ---------------------------------------------------------------- int8 product
PRODUCT = [(1, 1, 1), (1, 64, 64), (1, 4096, 1024), (2, 100, 300), (7, 129, 257), (16, 512, 4096), (17, 4096, 512),
           (33, 1000, 784), (48, 2048, 1024), (64, 256, 14336), (65, 640, 2000), (129, 384, 513), (200, 1008, 777),
           (256, 256, 256), (300, 5120, 1536), (333, 1024, 4096), (513, 192, 1023), (1000, 768, 2304),
           (2100, 512, 1100), (5000, 256, 320)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,m,n", PRODUCT)
def test_matmul_int8(T, m, n, dtype):
    xq, Wq = codes(21, T, m), codes(22, n, m)
    xs, ws = rnd(23, T).abs() + 0.01, rnd(24, n).abs() + 0.01
    z = px.matmul_int8(xq, xs, Wq, ws, dtype)
    want = (xq.double() @ Wq.double().t()) * xs.double()[:, None] * ws.double()
    within(z, want, (HALF[dtype] + 3.1 * U24) * want.abs(), "z")


def test_matmul_int8_largest_sums():
    # every product at its extreme over the longest contraction: exact in 32 bits
    m = 102400
    xq = torch.full((3, m), -128, dtype=torch.int8, device="cuda")
    Wq = torch.full((5, m), -128, dtype=torch.int8, device="cuda")
    Wq[1] = 127
    one = torch.ones(5, device="cuda")
    z = px.matmul_int8(xq, one[:3].contiguous(), Wq, one, F32)
    assert (z[:, 0] == 128 * 128 * m).all() and (z[:, 1] == -128 * 127 * m).all()


def test_matmul_int8_scales_carry_nan_and_zero():
    xq, Wq = codes(25, 4, 256), codes(26, 64, 256)
    xs, ws = torch.ones(4, device="cuda"), torch.ones(64, device="cuda")
    xs[1], xs[2], ws[5] = float("nan"), 0.0, float("nan")
    z = px.matmul_int8(xq, xs, Wq, ws, F32)
    assert torch.isnan(z[1]).all() and torch.isnan(z[:, 5]).all()
    rest = torch.ones(64, dtype=torch.bool)
    rest[5] = False
    assert not z[2, rest.cuda()].any() and torch.isfinite(z[0, rest.cuda()]).all()


def test_matmul_int8_leaves_what_lies_behind():
    # rows behind the last token and bytes around the output stay as they were
    T, m, n = 5, 256, 100
    xq, Wq, xs, ws = codes(27, T, m), codes(28, n, m), rnd(29, T).abs(), rnd(30, n).abs()
    for dtype, pd in ((BF, px.POETX_BF16), (F32, px.POETX_FP32)):
        big = torch.full((T + 3, n), 7.0, dtype=dtype, device="cuda")
        px.poetx_matmul_int8(T, n, m, xq, xs, Wq, ws, pd, big, None, 0)
        assert torch.equal(big[:T], px.matmul_int8(xq, xs, Wq, ws, dtype)) and (big[T:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,m,n", PRODUCT)
def test_matmul_int8_grad(T, m, n, dtype):
    dz, Wq, ws = rnd(31, T, n, dtype=dtype), codes(32, n, m), rnd(33, n).abs() + 0.01
    dx = px.matmul_int8_grad(dz, Wq, ws)
    q, s = quantise64(dz.float() * ws)
    want = (q @ Wq.double()) * s.double()[:, None]
    within(dx, want, (HALF[dtype] + 2.1 * U24) * want.abs(), "dx")


def test_matmul_int8_grad_is_near_the_exact_gradient():
    # against the unquantised formula: a code is off by at most half a scale, so a dx by at most
    # scale / 2 times the sum of |Wq| of its column
    T, m, n = 40, 320, 640
    dz, Wq, ws = rnd(34, T, n), codes(35, n, m), rnd(36, n).abs() + 0.01
    dx = px.matmul_int8_grad(dz, Wq, ws)
    u = dz.float() * ws
    _, s = quantise64(u)
    want = u.double() @ Wq.double()
    bound = 0.5 * s.double()[:, None] * Wq.double().abs().sum(0)
    within(dx, want, bound + 4 * U24 * (u.double().abs() @ Wq.double().abs()), "dx")


# ---------------------------------------------------------------- checkpoints
CKPT = [(1, 1), (1, 32), (3, 33), (5, 64), (17, 100), (300, 1001), (77, 1000), (130, 4096), (9, 14336), (2, 102400)]


def checkpoint64(x):
    """Values and biased exponents of a checkpoint, by the definition."""
    T, d = x.shape
    top = 127.0 * 2.0 ** 121
    w = torch.nn.functional.pad(x.double().clamp(-top, top), (0, -d % 32)).view(T, -1, 32)
    top = w.abs().amax(2)
    e = torch.full_like(top, -126.0)
    for k in range(-126, 121):  # the smallest e with top <= 127 * 2^e
        e = torch.where(top > 127.0 * 2.0 ** k, torch.full_like(e, float(k + 1)), e)
    bad = ~torch.isfinite(torch.nn.functional.pad(x, (0, -d % 32)).view(T, -1, 32)).all(2)
    step = torch.exp2(e)[:, :, None]
    v = ((w / step).round() * step).masked_fill(bad[:, :, None], float("nan")).view(T, -1)[:, :d]
    return v, (e + 127).masked_fill(bad, 255).to(torch.uint8)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", CKPT)
def test_checkpoint(T, d, dtype):
    x = rnd(37, T, d, dtype=dtype) * torch.exp2(torch.randint(-12, 12, (T, 1)).float()).cuda().to(dtype)
    c = px.checkpoint_save(x)
    v, e = checkpoint64(x)
    assert torch.equal(c.exps, e)
    for out in (BF, F32):
        assert torch.equal(px.checkpoint_load(c, out).double(), v)


def test_checkpoint_edges():
    # group maxima around every border of the exponent: 127 and 127.5 times a power of two, the
    # largest and smallest numbers, zeros
    rows = []
    for top in (127.0, 127.25, 127.5, 126.5, 128.0, 1.0, 2.0 ** -126, 2.0 ** -130, 2.0 ** -149, 3.38e38, 3.4028234e38, 3.37e38, 0.0,
                63.5, 2.0 ** -120 * 127, 2.0 ** -119 * 127.5):
        row = torch.linspace(-1, 1, 32) * top
        row[0], row[31] = -top, top
        rows.append(row)
    x = torch.stack(rows).cuda()
    c = px.checkpoint_save(x)
    v, e = checkpoint64(x)
    assert torch.equal(c.exps, e)
    within(px.checkpoint_load(c, F32), v, torch.zeros_like(v), "fp32")
    b = x.to(BF)  # (the largest fp32 number becomes an infinity here)
    c = px.checkpoint_save(b)
    v, e = checkpoint64(b)
    assert torch.equal(c.exps, e)
    within(px.checkpoint_load(c, BF), v, torch.zeros_like(v), "bf16")


@pytest.mark.parametrize("d", [96, 90])
def test_checkpoint_nonfinite_groups(d):
    x = rnd(38, 3, d, dtype=BF)
    x[0, 1], x[1, 40], x[2, d - 1] = float("inf"), float("nan"), -float("inf")
    v = px.checkpoint_load(px.checkpoint_save(x), F32)
    bad = torch.zeros(3, d, dtype=torch.bool)
    bad[0, :32] = bad[1, 32:64] = bad[2, 64:] = True
    assert torch.equal(torch.isnan(v).cpu(), bad)


BLOCK = [(BF, 1, 64, 64), (BF, 77, 192, 64), (BF, 300, 512, 128), (BF, 257, 1024, 256), (BF, 1, 256, 256),
         (BF, 1000, 768, 256), (BF, 2100, 256, 256), (BF, 5000, 2304, 256), (BF, 9001, 512, 256), (BF, 130, 1024, 512), (F32, 1, 2, 2), (F32, 65, 9, 3),
         (F32, 300, 512, 64), (F32, 1001, 80, 40), (F32, 40, 100, 100)]


@pytest.mark.parametrize("dtype,T,d,b", BLOCK)
def test_block_backward(dtype, T, d, b):
    x, D = rnd(39, T, d, dtype=dtype), rnd(40, T, d, dtype=dtype)
    G = rnd(41, d // b, b, b, dtype=dtype, scale=0.3)
    c = px.checkpoint_save(x)
    O, dG = px.block_backward(c, D, G)
    X = px.checkpoint_load(c, F32).double().view(T, d // b, b)
    D3, G3 = D.double().view(T, d // b, b), G.double()
    want_o = torch.einsum("tjc,jrc->tjr", D3, G3)
    size_o = torch.einsum("tjc,jrc->tjr", D3.abs(), G3.abs())
    # fp32 accumulation, a tensor-core addition cutting off up to a whole step: 2 u24 a term
    within(O.view(T, d // b, b), want_o, HALF[dtype] * want_o.abs() + 2 * (b + 2) * U24 * size_o, "O")
    want_g = torch.einsum("tjr,tjc->jrc", X, D3)
    tol_g = 2 * (T + 34) * U24 * torch.einsum("tjr,tjc->jrc", X.abs(), D3.abs())
    within(dG, want_g, tol_g, "dG")
    none, again = px.block_backward(c, D, G, need_o=False)
    assert none is None and torch.equal(again, dG)
    acc = torch.full_like(dG, 2.0)
    px.block_backward(c, D, G, dG=acc)
    within(acc, 2 + dG.double(), 2 * U24 * (2 + dG.double().abs()), "accumulated dG")


@pytest.mark.parametrize("power", [-110, -60, 90, 112, 119])
def test_block_backward_over_the_range_of_exponents(power):
    # checkpoints near both ends of the exponents' range, D scaled the other way: the products stay ordinary
    T, d, b = 300, 256, 256
    x = rnd(60, T, d) * 2.0 ** power
    D = (rnd(61, T, d) * 2.0 ** max(-110, -power)).to(BF)
    c = px.checkpoint_save(x)
    _, dG = px.block_backward(c, D, torch.zeros(1, b, b, dtype=BF, device="cuda"))
    X = px.checkpoint_load(c, F32).double()
    assert torch.isfinite(X).all()
    tol = 2 * (T + 34) * U24 * (X.abs().t() @ D.double().abs())
    within(dG[0], X.t() @ D.double(), tol, "dG")


def test_block_backward_nan_group_reaches_its_gradient():
    T, d, b = 40, 512, 256
    x, D, G = rnd(42, T, d, dtype=BF), rnd(43, T, d, dtype=BF), rnd(44, 2, b, b, dtype=BF)
    x[3, 300] = float("nan")
    _, dG = px.block_backward(px.checkpoint_save(x), D, G)
    bad = torch.isnan(dG)
    assert bad[1, 32:64].all() and not bad[0].any() and not bad[1, :32].any() and not bad[1, 64:].any()


# ---------------------------------------------------------------- empty batches
def test_empty_batches():
    e = torch.empty((0, 64), dtype=BF, device="cuda")
    q, s = px.quantize_rows(e)
    assert q.shape == (0, 64) and s.shape == (0,)
    g = torch.ones(64, device="cuda")
    assert px.rmsnorm_quantize(e, g, e, EPS).codes.shape == (0, 64)
    dx, dg = px.rmsnorm_backward(e, e, g, s)
    assert dx.shape == (0, 64) and not dg.any()
    keep = torch.full((64,), 3.0, device="cuda")
    px.rmsnorm_backward(e, e, g, s, dgamma=keep)
    assert (keep == 3).all()
    Wq, ws = codes(45, 32, 64), torch.ones(32, device="cuda")
    assert px.matmul_int8(q, s, Wq, ws).shape == (0, 32)
    assert px.matmul_int8_grad(torch.empty((0, 32), dtype=BF, device="cuda"), Wq, ws).shape == (0, 64)
    c = px.checkpoint_save(e)
    assert px.checkpoint_load(c, BF).shape == (0, 64)
    O, dG = px.block_backward(c, e, torch.ones(1, 64, 64, dtype=BF, device="cuda"))
    assert O.shape == (0, 64) and not dG.any()


# ---------------------------------------------------------------- offsets past 32 bits
def test_rows_past_two_to_the_31():
    # 150 001 rows of 14 336: 2.15e9 elements; the last rows against the same rows on their own
    T, d = 150_001, 14_336
    tail = rnd(70, 64, d, dtype=BF)
    x = torch.zeros(T, d, dtype=BF, device="cuda")
    x[-64:] = tail
    gamma = rnd(71, d) + 1

    def same(big, small):
        for a, b in zip(big, small):
            assert torch.equal(a[-64:], b)

    q = px.quantize_rows(x)
    same(q, px.quantize_rows(tail))
    assert not q.scale[:-64].any() and torch.equal(px.dequantize_rows(q.codes, q.scale, BF)[-64:],
                                                   px.dequantize_rows(q.codes[-64:].clone(), q.scale[-64:].clone(), BF))
    del q
    n, small = px.rmsnorm_quantize(x, gamma, x), px.rmsnorm_quantize(tail, gamma, tail)
    same(n[:4], small[:4])
    dx, dg = px.rmsnorm_backward(x, n.h, gamma, n.rstd)
    dx1, dg1 = px.rmsnorm_backward(tail, small.h, gamma, small.rstd)
    assert torch.equal(dx[-64:], dx1)
    # the other rows add nothing; 64 terms in another order
    assert ((dg - dg1).abs().double() <= 64 * U24 * (tail.double() * small.h.double() * small.rstd.double()[:, None]).abs().sum(0)).all()
    del n, dx
    c, c1 = px.checkpoint_save(x), px.checkpoint_save(tail)
    same(c, c1)
    assert torch.equal(px.checkpoint_load(c, BF)[-64:], px.checkpoint_load(c1, BF))
    G = rnd(72, d // 256, 256, 256, dtype=BF, scale=0.1)
    O, dG = px.block_backward(c, x, G)
    O1, dG1 = px.block_backward(c1, tail, G)
    assert torch.equal(O[-64:], O1) and not O[:-64].any()
    X = px.checkpoint_load(c1, F32).double().view(64, -1, 256)
    D = tail.double().view(64, -1, 256)
    assert ((dG - dG1).abs().double() <= 4 * 98 * U24 * torch.einsum("tjr,tjc->jrc", X.abs(), D.abs())).all()


@pytest.mark.parametrize("n", [14336, 14337])
def test_products_past_two_to_the_31(n):
    T, m = 150_001, 96
    xq, xs, Wq, ws = codes(73, T, m), rnd(74, T).abs(), codes(75, n, m), rnd(76, n).abs()
    z = px.matmul_int8(xq, xs, Wq, ws, BF)
    for part in (slice(0, 300), slice(T // 2, T // 2 + 300), slice(T - 300, T)):
        want = (xq[part].double() @ Wq.double().t()) * xs[part].double()[:, None] * ws.double()
        within(z[part], want, (HALF[BF] + 3.1 * U24) * want.abs(), "z")
    dx = px.matmul_int8_grad(z, Wq, ws)
    part = slice(T - 300, T)
    q, s = quantise64(z[part].float() * ws)
    want = (q @ Wq.double()) * s.double()[:, None]
    within(dx[part], want, (HALF[BF] + 2.1 * U24) * want.abs(), "dx")


# ---------------------------------------------------------------- together
def _chain_inputs(T, d, n):
    x, r = rnd(46, T, d, dtype=BF), rnd(47, T, d, dtype=BF)
    gamma = rnd(48, d, scale=0.1) + 1
    Wq, ws = codes(49, n, d), rnd(50, n).abs() * 1e-3 + 1e-4
    return x, r, gamma, Wq, ws, rnd(51, T, n, dtype=BF)


def _chain(x, r, gamma, Wq, ws, dz):
    """norm -> int8 product, and back: dz -> rows' gradient -> norm's gradient."""
    n = px.rmsnorm_quantize(x, gamma, r, EPS)
    z = px.matmul_int8(n.codes, n.scale, Wq, ws, BF)
    dy = px.matmul_int8_grad(dz, Wq, ws)
    dx, dg = px.rmsnorm_backward(dy, n.h, gamma, n.rstd, x)
    return z, dy, dx, dg


@pytest.mark.parametrize("T,d,n", [(1, 512, 768), (70, 1024, 640), (600, 512, 1280), (19, 1000, 333)])
def test_norm_product_and_back(T, d, n):
    x, r, gamma, Wq, ws, dz = _chain_inputs(T, d, n)
    z, dy, dx, dg = _chain(x, r, gamma, Wq, ws, dz)
    h = (x.float() + r.float()).to(BF)
    rs = (h.double().square().mean(1) + EPS).rsqrt()
    q, s = quantise64(h.float() * gamma)
    want = (q @ Wq.double().t()) * (s.double() * rs)[:, None] * ws.double()
    within(z, want, (2.0 ** -8 + (chain(d) + 5) * U24) * want.abs(), "z")
    gq, gs = quantise64(dz.float() * ws)
    want = (gq @ Wq.double()) * gs.double()[:, None]
    within(dy, want, (2.0 ** -8 + 2.1 * U24) * want.abs(), "dy")
    p, xn = dy.double() * gamma.double(), h.double() * rs[:, None]
    want = rs[:, None] * (p - xn * (p * xn).mean(1, keepdim=True)) + x.double()
    size = rs[:, None] * (p.abs() + xn.abs() * (p * xn).abs().mean(1, keepdim=True)) + x.double().abs()
    within(dx, want, 2.0 ** -8 * want.abs() + 4 * chain(d) * U24 * size, "dx")


def test_on_another_stream_and_in_a_graph():
    args = _chain_inputs(130, 512, 768)
    want = _chain(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _chain(*args)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two graphs of the same operators replayed at once on two streams, on new inputs
    statics = [[t.clone() for t in args] for _ in range(2)]
    graphs, outs = [], []
    for st in statics:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_chain(*st))
        graphs.append(g)
    new = [_chain_inputs(130, 512, 768), args]
    new[0] = [t.neg() if t.dtype == BF else t for t in new[0]]
    expect = [_chain(*n) for n in new]
    for st, n in zip(statics, new):
        for a, b in zip(st, n):
            a.copy_(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, e in zip(outs, expect):
        assert all(torch.equal(a, b) for a, b in zip(o, e))
