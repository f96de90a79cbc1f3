"""PoetxLinear in 8 bits: activations kept as checkpoints, the W0 product on
the int8 weight, and the served linear made of a trained layer.

Where a call is a sequence of operators that are tested on their own, it has to
give their bits; the token sums are compared with the checkpoints' own values in
64 bits (fp32 accumulation, up to a whole step cut off per addition: 2 u24 a
term, u24 = 2^-24)."""
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


def layer(m, n, b, dtype, sigma=0.02, seed=0):
    L = px.PoetxLinear(m, n, b, px.POETX_BF16 if dtype == BF else px.POETX_FP32)
    g = torch.Generator().manual_seed(100 + seed)
    tri = b * (b - 1) // 2
    L.load(rnd(101 + seed, n, m, dtype=dtype, scale=0.05), torch.randperm(m, generator=g).int().cuda(),
           torch.randperm(n, generator=g).int().cuda(), rnd(102 + seed, m // b, tri, scale=sigma),
           rnd(103 + seed, n // b, tri, scale=sigma))
    return L


def grads(L, x, saved, dz, need_dx=True):
    dGR = torch.full((L.m // L.b, L.b, L.b), float("nan"), device="cuda")
    dGP = torch.full((L.n // L.b, L.b, L.b), float("nan"), device="cuda")
    dx = L.backward_dG(x, saved, dz, dGR, dGP, need_dx=need_dx)
    return dx, dGR, dGP


CASES = [(BF, 512, 768, 256, 300), (BF, 256, 512, 256, 2100), (BF, 192, 320, 64, 77), (BF, 512, 1024, 512, 130),
         (F32, 192, 320, 64, 77), (F32, 40, 60, 20, 500), (F32, 9, 15, 3, 700), (BF, 512, 512, 256, 1)]


@pytest.mark.parametrize("dtype,m,n,b,T", CASES)
def test_checkpointed_layer(dtype, m, n, b, T):
    L = layer(m, n, b, dtype)
    x, dz = rnd(1, T, m, dtype=dtype), rnd(2, T, n, dtype=dtype)
    z, plain = L.forward(x, save_xg=True)
    z8, kept = L.forward(x, save_xg=True, save8=True)
    assert torch.equal(z8, z)
    for k, p in zip(kept, plain):
        c = px.checkpoint_save(p)
        assert torch.equal(k.codes, c.codes) and torch.equal(k.exps, c.exps)
    dx, dGR, dGP = grads(L, None, plain, dz)
    dx8, dGR8, dGP8 = grads(L, None, kept, dz)
    # O = D G^T is the same product of the same operands, summed over b terms
    tol = 2.0 ** -7 if dtype == BF else 1e-5
    assert ((dx8 - dx).double().norm() <= tol * dx.double().norm())
    # P side: dV = dz in the Psi_P frame, Y as kept
    dV = dz[:, L.permP.long()].double().view(T, n // b, b)
    Y = px.checkpoint_load(kept.y, F32).double().view(T, n // b, b)
    want = torch.einsum("tjr,tjc->jrc", Y, dV)
    bound = 2 * (T + 34) * U24 * torch.einsum("tjr,tjc->jrc", Y.abs(), dV.abs())
    assert ((dGP8.double() - want).abs() <= bound).all()
    # R side: the plain backward given the expanded checkpoint sees the same values
    ref = px.Saved(px.checkpoint_load(kept.y, dtype), px.checkpoint_load(kept.xg, dtype))
    _, rR, rP = grads(L, None, ref, dz)
    for got, r in ((dGR8, rR), (dGP8, rP)):
        # two fp32 sums of the same T products: each off by 2 (T + 34) u24 of the sum of magnitudes, which
        # Cauchy-Schwarz bounds by the operands' norms; checked on the whole block array
        assert (got - r).double().norm() <= 1e-5 * r.double().norm() + 1e-30
    # a backward from x (no Xg kept), with a dz only for the triangles, accumulated
    dq1 = L.backward(x, px.Saved(kept.y, None), dz)
    dq2 = L.backward(x, kept.y, dz, need_dx=False)
    assert dq2[0] is None and torch.equal(dq1[1], dq2[1]) and torch.equal(dq1[2], dq2[2])
    acc = [dq1[1].clone(), dq1[2].clone()]
    L.backward(x, kept.y, dz, dqR=acc[0], dqP=acc[1], accumulate=True)
    for a, d in zip(acc, dq1[1:]):
        assert torch.allclose(a, 2 * d, rtol=1e-6, atol=0)


def test_recompute_from_a_checkpointed_input():
    # nothing kept but Xg in 8 bits: Y is recomputed from its values
    L = layer(256, 512, 256, BF)
    x, dz = rnd(3, 200, 256, dtype=BF), rnd(4, 200, 512, dtype=BF)
    _, kept = L.forward(x, save_xg=True, save8=True)
    xg = px.checkpoint_load(kept.xg, BF)
    a = grads(L, None, px.Saved(None, kept.xg), dz)
    b = grads(L, None, px.Saved(None, xg), dz)
    for s, t in zip(a, b):
        assert (s.double() - t.double()).norm() <= 1e-5 * t.double().norm()


@pytest.mark.parametrize("dtype,m,n,b,T", [(BF, 512, 768, 256, 300), (BF, 192, 320, 64, 33), (F32, 60, 90, 30, 50),
                                           (BF, 512, 512, 512, 1), (F32, 64, 128, 64, 600)])
def test_int8_weight_product_is_the_operators_sequence(dtype, m, n, b, T):
    L = layer(m, n, b, dtype, sigma=0.0)       # G = I: U = Xg and dY = dV, so every operand can be seen
    x, dz = rnd(5, T, m, dtype=dtype), rnd(6, T, n, dtype=dtype)
    L.quantize_weight(int8_product=True)
    z, saved = L.forward(x, save_xg=True)
    rows = px.quantize_rows(x[:, L.permR.long()].contiguous())
    Y = px.matmul_int8(rows.codes, rows.scale, L.Wq, L.Wscale, dtype)
    assert torch.equal(saved.y, Y)
    assert torch.equal(z[:, L.permP.long()], Y)
    dU = px.matmul_int8_grad(dz[:, L.permP.long()].contiguous(), L.Wq, L.Wscale)
    for s in (saved, None):                    # kept, and recomputed
        dx, dqR, dqP = L.backward(x, s, dz)
        assert torch.equal(dx[:, L.permR.long()], dU)
        if s is not None:
            first = dqR, dqP
    assert torch.equal(first[0], dqR) and torch.equal(first[1], dqP)
    # with checkpoints as well
    z8, kept = L.forward(x, save_xg=True, save8=True)
    assert torch.equal(z8, z)
    dx8, _, _ = L.backward(None, kept, dz)
    assert torch.equal(dx8[:, L.permR.long()], dU)
    with pytest.raises(RuntimeError, match="merge"):
        L.merge(L.permR, L.permP)
    with pytest.raises(RuntimeError, match="export_weight"):
        L.export_weight()
    with pytest.raises(RuntimeError, match="abi"):
        L.abi()
    with pytest.raises(RuntimeError, match="quantize_weight"):
        L.quantize_weight()
    px.LayerGroup([L]).build()                 # the blocks are still built
    W0 = rnd(7, n, m, dtype=dtype)
    L.load(W0, L.permR.clone(), L.permP.clone(), L.qR.clone(), L.qP.clone())   # and a new weight is a weight
    assert not L.int8_product and torch.equal(L.export_weight(), W0)


def test_int8_weight_product_is_near_the_bf16_layer():
    # a code is off by half a scale of its row, scale = max / 127; over K = 1024 terms of independent signs
    # the product's relative error is about sqrt(ex^2 + ew^2), e = (max / rms) / (127 sqrt(12)) of a row,
    # with max / rms below 4.5 in normal rows this long: 1.5 %
    L = layer(1024, 1024, 256, BF)
    x, dz = rnd(7, 256, 1024, dtype=BF), rnd(8, 256, 1024, dtype=BF)
    z, s = L.forward(x, save_xg=True)
    dx, dqR, dqP = L.backward(x, s, dz)
    L.quantize_weight(int8_product=True)
    z8, s8 = L.forward(x, save_xg=True)
    dx8, dqR8, dqP8 = L.backward(x, s8, dz)
    for a, b in ((z8, z), (dx8, dx)):
        assert (a - b).double().norm() <= 0.02 * b.double().norm()
    for a, b in ((dqR8, dqR), (dqP8, dqP)):
        assert (a - b).double().norm() <= 0.05 * b.double().norm()


def test_served_linear_of_a_trained_layer():
    L = layer(512, 768, 256, BF)
    before = [t.clone() for t in (L.W, L.qR, L.qP, L.GR, L.GP)]
    lin = px.Int8Linear.from_layer(L)
    for a, b in zip(before, (L.W, L.qR, L.qP, L.GR, L.GP)):
        assert torch.equal(a, b)
    gamma = rnd(9, 512, scale=0.1) + 1
    for T in (1, 40, 400):
        x, r = rnd(10 + T, T, 512, dtype=BF), rnd(11 + T, T, 512, dtype=BF)
        n = px.rmsnorm_quantize(x, gamma, r, y=True)
        z = lin.forward(n)
        want, _ = L.forward(n.y, save=False)
        # the weight's and the tokens' codes: 1.5 % as above, and the layer's own bf16 roundings
        assert (z - want).double().norm() <= 0.03 * want.double().norm()
        assert torch.equal(z, px.matmul_int8(n.codes, n.scale, lin.Wq, lin.wscale, BF))
        q = px.quantize_rows(n.y)
        assert torch.equal(lin.forward(n.y), lin.forward(q))
        assert torch.equal(lin.backward(z), px.matmul_int8_grad(z, lin.Wq, lin.wscale))


def test_training_step_in_eight_bits():
    """Norm, layer with the int8 weight and checkpoints, and back: a captured
    step replays to the eager step's bits, and its gradients are near those of
    the same step in bf16."""
    T, m, n = 300, 512, 768
    x, r, dz, gamma = rnd(20, T, m, dtype=BF), rnd(21, T, m, dtype=BF), rnd(22, T, n, dtype=BF), rnd(23, m) * 0.1 + 1
    L = layer(m, n, 256, BF)

    def step(save8):
        h = px.rmsnorm_quantize(x, gamma, r, codes=False, y=True)
        z, saved = L.forward(h.y, save_xg=True, save8=save8)
        dy, dqR, dqP = L.backward(None, saved, dz)
        dx, dg = px.rmsnorm_backward(dy, h.h, gamma, h.rstd)
        return z, dqR, dqP, dx, dg

    want = step(False)
    L.quantize_weight(int8_product=True)
    eager = step(True)
    for a, b in zip(eager, want):
        assert (a - b).double().norm() <= 0.05 * b.double().norm()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(True)
    for t in out:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_graphs_of_one_layer_hold_their_own_workspaces():
    # two captured steps of one layer replayed on two streams at once, after an eager call that needed a
    # larger workspace than either
    L = layer(512, 768, 256, BF)
    ins = [(rnd(30 + i, T, 512, dtype=BF), rnd(40 + i, T, 768, dtype=BF)) for i, T in enumerate((300, 200))]

    def step(x, dz):
        z, saved = L.forward(x, save_xg=True, save8=True)
        return (z, *L.backward(None, saved, dz))

    want = [step(*a) for a in ins]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*a))
        graphs.append(g)
    step(rnd(50, 900, 512, dtype=BF), rnd(51, 900, 768, dtype=BF))
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(bool(torch.isnan(j).all()) for j in junk)
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_empty_batch():
    L = layer(256, 512, 256, BF)
    x, dz = torch.empty(0, 256, dtype=BF, device="cuda"), torch.empty(0, 512, dtype=BF, device="cuda")
    for _ in range(2):
        z, kept = L.forward(x, save_xg=True, save8=True)
        assert z.shape == (0, 512)
        dx, dqR, dqP = L.backward(None, kept, dz)
        assert dx.shape == (0, 256) and not dqR.any() and not dqP.any()
        if not L.int8_product:
            L.quantize_weight(int8_product=True)


def test_refusals_of_the_layer():
    L = px.PoetxLinear(256, 256, 64, px.POETX_BF16, fold=px.POETX_FOLD_ALL)
    x = torch.zeros(4, 256, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="save8"):
        L.forward(x, save8=True)
    with pytest.raises(ValueError, match="int8_product"):
        L.quantize_weight(int8_product=True)
    L = px.PoetxLinear(256, 256, 64, px.POETX_BF16)
    c = px.checkpoint_save(x)
    with pytest.raises(TypeError, match="y: expected a Checkpoint"):
        L.forward(x, save8=True, y=x)
    with pytest.raises(TypeError, match="y: expected a torch.Tensor"):
        L.forward(x, y=c)
    with pytest.raises(ValueError, match="saved y codes: shape"):
        L.backward(x, px.Checkpoint(c.codes[:3], c.exps[:3]), x)
    with pytest.raises(ValueError, match="saved y exps: shape"):
        L.backward(x, px.Checkpoint(c.codes, c.exps[:, :7].contiguous()), x)
    with pytest.raises(px.PoetxError) as e:  # a checkpoint and a tensor of the same activation
        nb = px.poetx_backward_recompute_workspace_bytes(L.abi(), 4) + (1 << 20)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        px.poetx_backward_q8(L.abi(), 4, x, x, None, px.make_q8(y_codes=c.codes, y_exps=c.exps), x, None, L.qR, L.qP, 0,
                             ws, nb)
    assert e.value.status == 1


def test_other_device_than_the_current_one():
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    with torch.cuda.device(1):
        x = torch.randn(4, 64, device="cuda:1").to(BF)
    q = px.quantize_rows(x)
    assert q.codes.device == x.device
