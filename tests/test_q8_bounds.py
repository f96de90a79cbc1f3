"""The 8-bit operators inside larger buffers, and behind other work: what lies
around an output stays as it was, what lies around an input is not seen, and a
call waits for whatever wrote its inputs, in a stream and in a graph."""
import pytest
import torch

import orthogonal_equivalence_b200 as px
from orthogonal_equivalence_b200 import build as pbuild

pytestmark = pytest.mark.gpu

BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
DT = {BF: px.POETX_BF16, F32: px.POETX_FP32}


@pytest.fixture(scope="module", autouse=True)
def library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pbuild.build()
    px.lib()
    px.poetx_device_error()
    yield
    torch.cuda.synchronize()
    assert px.poetx_device_error() == 0


def rnd(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


class Around:
    """Tensors between two margins of one buffer each, filled with a byte that reads as NaN (0xff) or as 127 (0x7f)."""
    MARGIN = 64 * 1024

    def __init__(self, byte):
        self.byte, self.held = byte, []

    def like(self, t, fill=True):
        n = t.numel() * t.element_size()
        raw = torch.full((2 * self.MARGIN + n + 64,), self.byte, dtype=torch.uint8, device="cuda")
        at = raw[self.MARGIN:self.MARGIN + n].view(t.dtype).view(t.shape)
        if fill:
            at.copy_(t)
        self.held.append((raw, n))
        return at

    def out(self, *shape, dtype):
        return self.like(torch.empty(*shape, dtype=dtype, device="cuda"), fill=False)

    def untouched(self):
        return all(bool((raw[:self.MARGIN] == self.byte).all()) and bool((raw[self.MARGIN + n:] == self.byte).all())
                   for raw, n in self.held)


SIZES = [(1, 64), (5, 4096), (37, 192), (300, 1001), (259, 2261), (7, 14336), (700, 640), (1300, 1025), (3, 33)]


@pytest.mark.parametrize("byte", [0xff, 0x7f])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", SIZES)
def test_rows_between_margins(T, d, dtype, byte):
    A, pd = Around(byte), DT[dtype]
    x, r, gamma = rnd(1, T, d, dtype=dtype), rnd(2, T, d, dtype=dtype), rnd(3, d) + 1
    ax, ar, ag = A.like(x), A.like(r), A.like(gamma)
    q, s = A.out(T, d, dtype=I8), A.out(T, dtype=F32)
    px.poetx_quantize_rows(T, d, ax, pd, ag, q, s)
    for a, w in zip((q, s), px.quantize_rows(x, gamma)):
        assert torch.equal(a, w)
    h, y, rstd = A.out(T, d, dtype=dtype), A.out(T, d, dtype=dtype), A.out(T, dtype=F32)
    q, s = A.out(T, d, dtype=I8), A.out(T, dtype=F32)
    px.poetx_rmsnorm_quantize(T, d, ax, ar, ag, 1e-5, pd, h, y, q, s, rstd)
    n = px.rmsnorm_quantize(x, gamma, r, 1e-5, y=True)
    for a, w in zip((q, s, h, rstd, y), n):
        assert torch.equal(a, w)
    dx, dg = A.out(T, d, dtype=dtype), A.out(d, dtype=F32)
    nb = px.poetx_rmsnorm_backward_workspace_bytes(T, d, pd)
    px.poetx_rmsnorm_backward(T, d, ax, A.like(n.h), ag, A.like(n.rstd), ar, pd, dx, dg, 0,
                              A.out(nb, dtype=torch.uint8), nb)
    for a, w in zip((dx, dg), px.rmsnorm_backward(x, n.h, gamma, n.rstd, r)):
        assert torch.equal(a, w)
    c, e = A.out(T, d, dtype=I8), A.out(T, (d + 31) // 32, dtype=torch.uint8)
    px.poetx_checkpoint_save(T, d, ax, pd, c, e)
    kept = px.checkpoint_save(x)
    assert torch.equal(c, kept.codes) and torch.equal(e, kept.exps)
    back = A.out(T, d, dtype=dtype)
    px.poetx_checkpoint_load(T, d, A.like(c), A.like(e), pd, back)
    assert torch.equal(back, px.checkpoint_load(kept, dtype))
    w = A.out(T, d, dtype=dtype)
    px.poetx_weight_dequantize(T, d, A.like(q), A.like(s), pd, w)
    assert torch.equal(w, px.dequantize_rows(q, s, dtype))
    assert A.untouched()


@pytest.mark.parametrize("byte", [0xff, 0x7f])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,m,n", [(1, 64, 64), (1, 4096, 1000), (17, 1008, 777), (100, 333, 513), (130, 256, 96), (700, 512, 1023),
                                   (2100, 520, 1100), (333, 40, 2049)])
def test_products_between_margins(T, m, n, dtype, byte):
    A, pd = Around(byte), DT[dtype]
    g = torch.Generator().manual_seed(5)
    xq = torch.randint(-128, 128, (T, m), generator=g, dtype=I8).cuda()
    Wq = torch.randint(-128, 128, (n, m), generator=g, dtype=I8).cuda()
    xs, ws = rnd(6, T).abs() + 0.01, rnd(7, n).abs() + 0.01
    z, aW, aws = A.out(T, n, dtype=dtype), A.like(Wq), A.like(ws)
    nb = px.poetx_matmul_int8_workspace_bytes(T, n, m)
    px.poetx_matmul_int8(T, n, m, A.like(xq), A.like(xs), aW, aws, pd, z, A.out(nb, dtype=torch.uint8), nb)
    assert torch.equal(z, px.matmul_int8(xq, xs, Wq, ws, dtype))
    dx = A.out(T, m, dtype=dtype)
    nb = px.poetx_matmul_int8_grad_workspace_bytes(T, n, m)
    px.poetx_matmul_int8_grad(T, n, m, A.like(z), aW, aws, pd, dx, A.out(nb, dtype=torch.uint8), nb)
    assert torch.equal(dx, px.matmul_int8_grad(z, Wq, ws))
    assert A.untouched()


@pytest.mark.parametrize("byte", [0xff, 0x7f])
@pytest.mark.parametrize("dtype,T,d,b", [(BF, 1, 64, 64), (BF, 77, 192, 64), (BF, 300, 512, 128), (BF, 257, 1024, 256), (BF, 2300, 512, 256),
                                         (BF, 1, 256, 256), (BF, 130, 1024, 512), (F32, 65, 9, 3), (F32, 300, 512, 64), (F32, 1001, 80, 40),
                                         (F32, 33, 100, 50)])
def test_blocks_between_margins(dtype, T, d, b, byte):
    A, pd = Around(byte), DT[dtype]
    c = px.checkpoint_save(rnd(8, T, d, dtype=dtype))
    D, G = rnd(9, T, d, dtype=dtype), rnd(10, d // b, b, b, dtype=dtype)
    O, dG = A.out(T, d, dtype=dtype), A.out(d // b, b, b, dtype=F32)
    nb = px.poetx_block_backward_workspace_bytes(T, d, b, pd)
    px.poetx_block_backward(T, d, b, A.like(c.codes), A.like(c.exps), A.like(D), A.like(G), pd, O, dG, 0,
                            A.out(nb, dtype=torch.uint8), nb)
    for a, w in zip((O, dG), px.block_backward(c, D, G)):
        assert torch.equal(a, w)
    assert A.untouched()


# ---------------------------------------------------------------- behind other work
# The product of few tokens starts while the kernel before it ends, so all it reads has to have been waited for:
# work of another stream (an event between the two), a copy and a fill (no kernels), and a kernel.
def _inputs(seed, T=3, m=1024, n=2048):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(-128, 128, (T, m), generator=g, dtype=I8).cuda(), rnd(seed, T).abs(),
            torch.randint(-128, 128, (n, m), generator=g, dtype=I8).cuda(), rnd(seed + 1, n).abs()]


def _steps(bufs, new, side, busy):
    """Products behind a join, behind a copy, behind a fill and behind a kernel, each reading what came right before."""
    here = torch.cuda.current_stream()
    outs = []
    x, xs, W, ws = bufs
    for b in bufs:                      # (the last replay's end)
        b.zero_()
    side.wait_stream(here)
    with torch.cuda.stream(side):
        if busy:
            torch.cuda._sleep(2_000_000)
        for b, n in zip(bufs, new):
            b.copy_(n)
    px.matmul_int8(new[0], new[1], new[2], new[3])      # a product before the join, to follow closely
    here.wait_stream(side)
    outs.append(px.matmul_int8(*bufs))
    x.copy_(new[0].flip(0))
    outs.append(px.matmul_int8(*bufs))
    x.zero_()
    outs.append(px.matmul_int8(*bufs))
    torch.add(new[0], 0, out=x)
    torch.mul(new[3], 2, out=ws)
    outs.append(px.matmul_int8(*bufs))
    xs.copy_(new[1].flip(0))
    outs.append(px.matmul_int8(*bufs))
    return outs


def _expected(new):
    x, xs, W, ws = new
    return [px.matmul_int8(*a) for a in ((x, xs, W, ws), (x.flip(0), xs, W, ws), (x * 0, xs, W, ws), (x, xs, W, 2 * ws),
                                         (x, xs.flip(0), W, 2 * ws))]


def test_products_wait_for_what_comes_before_them():
    new = _inputs(20)
    want = _expected(new)
    bufs, side = [torch.zeros_like(t) for t in new], torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        outs = _steps(bufs, new, side, busy=True)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    for o in outs:
        o.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = _steps(bufs, new, side, busy=True)
    for i in range(20):
        for t, n in zip(new, _inputs(30 + i % 3)):
            t.copy_(n)
        want = _expected(new)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


# ---------------------------------------------------------------- the layer
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("dtype,m,n,b,T", [(BF, 512, 768, 256, 300), (BF, 192, 320, 64, 2100), (BF, 512, 1024, 512, 130), (F32, 40, 60, 20, 500),
                                           (F32, 9, 15, 3, 70), (BF, 256, 256, 256, 1)])
def test_a_layer_between_margins(dtype, m, n, b, T, i8):
    # every form of what is kept: scratch of exactly the size asked for, its bytes read as NaN
    pd, tri = DT[dtype], b * (b - 1) // 2
    L = px.PoetxLinear(m, n, b, pd)
    g = torch.Generator().manual_seed(1)
    L.load(rnd(1, n, m, dtype=dtype) * 0.05, torch.randperm(m, generator=g).int().cuda(),
           torch.randperm(n, generator=g).int().cuda(), rnd(2, m // b, tri) * 0.02, rnd(3, n // b, tri) * 0.02)
    abi = L.abi()
    wq = {}
    if i8:
        Wq, ws = torch.empty(n, m, dtype=I8, device="cuda"), torch.empty(n, device="cuda")
        px.poetx_weight_quantize(n, m, L.W, pd, Wq, ws)
        wq = {"Wq": Wq, "wscale": ws}
    x, dz = rnd(4, T, m, dtype=dtype), rnd(5, T, n, dtype=dtype)

    def run(A, exact, y, xg):
        """z, what is kept and the gradients; y and xg: None, "full" or "codes"."""
        out = A.out if A else lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")
        take = A.like if A else lambda t: t

        def scratch(nbytes):
            nbytes += 0 if exact else 1 << 22
            return out(nbytes, dtype=torch.uint8), nbytes

        def keep(form, d):
            return (out(T, d, dtype=dtype) if form == "full" else None,
                    (out(T, d, dtype=I8), out(T, (d + 31) // 32, dtype=torch.uint8)) if form == "codes" else (None, None))

        ys, yc = keep(y, n)
        xs, xc = keep(xg, m)
        q = px.make_q8(**wq, y_codes=yc[0], y_exps=yc[1], xg_codes=xc[0], xg_exps=xc[1])
        z, dx = out(T, n, dtype=dtype), out(T, m, dtype=dtype)
        ax, adz = take(x), take(dz)
        px.poetx_forward_q8(abi, T, ax, z, ys, xs, q, *scratch(px.poetx_forward_q8_workspace_bytes(abi, T, q)))
        nb = px.poetx_backward_q8_workspace_bytes(abi, T, int(ys is not None), q)
        dqR, dqP = out(m // b, tri, dtype=F32), out(n // b, tri, dtype=F32)
        px.poetx_backward_q8(abi, T, ax, ys, xs, q, adz, dx, dqR, dqP, 0, *scratch(nb))
        dGR, dGP = out(m // b, b, b, dtype=F32), out(n // b, b, b, dtype=F32)
        px.poetx_backward_dG_q8(abi, T, ax, ys, xs, q, adz, None, dGR, dGP, 0, *scratch(nb))
        kept = [t for t in (ys, xs, *yc, *xc) if t is not None]
        return [z, dx, dqR, dqP, dGR, dGP] + kept

    for y in (None, "full", "codes"):
        for xg in (None, "full", "codes"):
            A = Around(0xff)
            got, want = run(A, True, y, xg), run(None, False, y, xg)
            assert all(torch.equal(a, w) for a, w in zip(got, want)), (y, xg)
            assert A.untouched(), (y, xg)
