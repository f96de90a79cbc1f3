"""A layer that changes between its forms: its weight in full, as int8 codes
expanded before use (a scratch that several layers share), and as int8 codes
that the W0 product multiplies.  Each change and each call of the weight has
to see the layer's own weight, whatever the scratch holds."""
import pytest
import torch

import orthogonal_equivalence_b200 as px
from orthogonal_equivalence_b200 import build as pbuild

pytestmark = pytest.mark.gpu

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


def state(m, n, b, dtype, seed):
    """(W0, permR, permP, qR, qP) as PoetxLinear.load takes them."""
    g = torch.Generator().manual_seed(100 + seed)
    tri = b * (b - 1) // 2
    return (rnd(101 + seed, n, m, dtype=dtype, scale=0.05), torch.randperm(m, generator=g).int().cuda(),
            torch.randperm(n, generator=g).int().cuda(), rnd(102 + seed, m // b, tri, scale=0.02),
            rnd(103 + seed, n // b, tri, scale=0.02))


def layer(m, n, b, dtype, st):
    L = px.PoetxLinear(m, n, b, px.POETX_BF16 if dtype == BF else px.POETX_FP32)
    L.load(*st)
    return L


def two_on_one_scratch(m, n, b, dtype):
    """A POET-XQ layer whose scratch another layer has used since, the states of both, and the other layer."""
    st, other = state(m, n, b, dtype, 0), state(m, n, b, dtype, 50)
    A, B = layer(m, n, b, dtype, st), layer(m, n, b, dtype, other)
    scratch = torch.full((n * m,), float("nan"), dtype=dtype, device="cuda")
    A.quantize_weight(scratch)
    B.quantize_weight(scratch)
    B.forward(rnd(9, 3, m, dtype=dtype))
    return A, st, B, other


FORMS = [(BF, 512, 768, 256, 70), (F32, 60, 90, 30, 50)]


@pytest.mark.parametrize("dtype,m,n,b,T", FORMS)
def test_a_new_weight_of_a_quantized_layer(dtype, m, n, b, T):
    A, _, _, _ = two_on_one_scratch(m, n, b, dtype)
    new = state(m, n, b, dtype, 80)
    x, dz = rnd(1, T, m, dtype=dtype), rnd(2, T, n, dtype=dtype)
    full = layer(m, n, b, dtype, new)
    A.load(*new)
    assert A.Wq is None and torch.equal(A.export_weight(), new[0])
    for _ in range(2):      # in full, and quantized again
        z, saved = full.forward(x)
        z8, saved8 = A.forward(x)
        assert torch.equal(z8, z)
        for got, want in zip(A.backward(x, saved8, dz), full.backward(x, saved, dz)):
            assert torch.equal(got, want)
        if A.Wq is None:
            A.quantize_weight()
            full.quantize_weight()


def expanded(W0):
    """A natural weight after its rows went through int8 codes (a row keeps its
    scale under any order of its columns)."""
    n, m = W0.shape
    q, s = torch.empty(n, m, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    px.poetx_weight_quantize(n, m, W0, px.POETX_BF16 if W0.dtype == BF else px.POETX_FP32, q, s)
    return px.dequantize_rows(q, s, W0.dtype)


@pytest.mark.parametrize("dtype,m,n,b,T", FORMS)
def test_a_quantized_layer_takes_the_int8_product(dtype, m, n, b, T):
    A, st, _, _ = two_on_one_scratch(m, n, b, dtype)
    direct = layer(m, n, b, dtype, st)
    direct.quantize_weight(int8_product=True)
    A.quantize_weight(int8_product=True)
    assert torch.equal(A.Wq, direct.Wq) and torch.equal(A.Wscale, direct.Wscale)
    x, dz = rnd(1, T, m, dtype=dtype), rnd(2, T, n, dtype=dtype)
    for got, want in zip(A.backward(x, A.forward(x)[1], dz), direct.backward(x, direct.forward(x)[1], dz)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,m,n,b,T", FORMS)
def test_a_quantized_layer_takes_another_scratch(dtype, m, n, b, T):
    A, st, _, _ = two_on_one_scratch(m, n, b, dtype)
    codes, scale = A.Wq.clone(), A.Wscale.clone()
    A.quantize_weight()
    assert torch.equal(A.Wq, codes) and torch.equal(A.Wscale, scale)
    x = rnd(1, T, m, dtype=dtype)
    want = layer(m, n, b, dtype, (expanded(st[0]), *st[1:])).forward(x)[0]
    assert torch.equal(A.forward(x)[0], want)


@pytest.mark.parametrize("dtype,m,n,b,T", FORMS)
def test_the_weight_of_a_quantized_layer_is_exported(dtype, m, n, b, T):
    A, st, B, other = two_on_one_scratch(m, n, b, dtype)
    for L, s in ((A, st), (B, other), (A, st)):
        assert torch.equal(L.export_weight(), expanded(s[0]))


@pytest.mark.parametrize("dtype,m,n,b,T", FORMS)
def test_a_quantized_layer_is_merged(dtype, m, n, b, T):
    A, st, B, other = two_on_one_scratch(m, n, b, dtype)
    new = state(m, n, b, dtype, 80)[1:3]
    x, dz = rnd(1, T, m, dtype=dtype), rnd(2, T, n, dtype=dtype)
    for L, s in ((A, st), (B, other)):
        full = layer(m, n, b, dtype, (expanded(s[0]), *s[1:]))
        full.merge(*new)
        merged = full.W.clone()
        full.quantize_weight()
        L.merge(*new)
        assert torch.equal(L.Wq, full.Wq) and torch.equal(L.Wscale, full.Wscale)
        assert torch.equal(L.permR, new[0]) and torch.equal(L.permP, new[1]) and not L.qR.any() and not L.qP.any()
        # what the codes stand for is the merged weight to half a step, and the bf16 rounding of that
        assert ((L.export_weight()[new[1].long()][:, new[0].long()].double() - merged.double()).abs() <=
                (0.5 + 127 * 2.0 ** -8) * L.Wscale.double()[:, None] * (1 + 1e-6)).all()
    for L, s in ((A, st), (B, other)):
        z, saved = L.forward(x)
        W = px.dequantize_rows(L.Wq, L.Wscale, dtype)          # in the frame: G = I and z = Xg W^T there
        want = x[:, new[0].long()].double() @ W.double().t()
        size = x[:, new[0].long()].double().abs() @ W.double().abs().t()
        # m fp32 sums (up to a whole step each on the tensor cores), one rounding to dtype
        half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
        assert ((z[:, new[1].long()].double() - want).abs() <= half * want.abs() + 2 * (m + 2) * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("handle", [False, True])
def test_a_served_linear_made_on_another_stream(handle, quantized):
    # either stream is kept busy in turn, so that work that is not ordered between the two would be seen: the
    # layer's last change is still to come on the current stream, and memory that the call gives back is used there
    m, n, b = 512, 768, 256
    st = state(m, n, b, BF, 0)
    L = layer(m, n, b, BF, st)
    if quantized:
        L.quantize_weight()
    want = px.Int8Linear.from_layer(L)
    L.qR.zero_()
    L.build()
    side = torch.cuda.Stream()
    for _ in range(2):                   # (the second one finds the allocator's memory used)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        L.qR.copy_(st[3])
        L.build()
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)
        lin = px.Int8Linear.from_layer(L, stream=side.cuda_stream if handle else side)
        junk = [torch.full((s,), 77, dtype=torch.uint8, device="cuda") for s in (m * n * 2, m * n * 8, m * 4, n * 4) * 4]
        got = lin.Wq.clone(), lin.wscale.clone()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want.Wq) and torch.equal(got[1], want.wscale)
        assert all(bool((j == 77).all()) for j in junk)
        L.qR.zero_()
        L.build()


def test_a_served_linear_made_on_the_default_stream_from_another():
    L = layer(512, 768, 256, BF, state(512, 768, 256, BF, 0))
    want = px.Int8Linear.from_layer(L)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lin = px.Int8Linear.from_layer(L, stream=0)
        same = torch.equal(lin.Wq, want.Wq) and torch.equal(lin.wscale, want.wscale)
    assert same


@pytest.mark.parametrize("int8_product", [False, True])
def test_two_layers_on_two_streams_of_one_graph(int8_product):
    # a graph that forks: one layer on a given stream, the other on the graph's own, with nothing between them
    # but the join, and scratch of the same sizes
    T, m, n = 700, 512, 768
    layers = [layer(m, n, 256, BF, state(m, n, 256, BF, 30 * i)) for i in range(2)]
    ins = [(rnd(1 + i, T, m, dtype=BF), rnd(11 + i, T, n, dtype=BF)) for i in range(2)]
    if int8_product:
        for L in layers:
            L.quantize_weight(int8_product=True)

    def step(i, stream=None):
        x, dz = ins[i]
        z, saved = layers[i].forward(x, save_xg=True, stream=stream)
        return (z, *layers[i].backward(None, saved, dz, stream=stream)), saved

    want = [step(i)[0] for i in range(2)]
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        out = [None, None]
        out[0], held = step(0, side)     # (what the caller holds, it holds until the join)
        out[1], _ = step(1)
        here.wait_stream(side)
        del held
    for _ in range(4):
        for o in out:
            for t in o:
                t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(out, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_load_merge_and_quantize_on_another_stream():
    # the current stream is busy: what these calls do with torch has to go to the stream they are given, too
    m, n, b = 512, 768, 256
    first, st, new = state(m, n, b, BF, 0), state(m, n, b, BF, 50), state(m, n, b, BF, 80)[1:3]
    x = rnd(1, 40, m, dtype=BF)
    full = layer(m, n, b, BF, st)
    full.merge(*new)
    want = full.forward(x)[0]
    full.quantize_weight()
    want8 = full.forward(x)[0]
    L, side = layer(m, n, b, BF, first), torch.cuda.Stream()
    new64 = [p.long() for p in new]       # (converted by the call)
    torch.cuda.synchronize()
    torch.cuda._sleep(60_000_000)
    L.load(*st, stream=side)
    L.merge(*new64, stream=side)
    z = L.forward(x, stream=side)[0]
    L.quantize_weight(stream=side)
    z8 = L.forward(x, stream=side)[0]
    side.synchronize()
    with torch.cuda.stream(side):
        same = torch.equal(z, want), torch.equal(z8, want8), torch.equal(L.Wq, full.Wq)
    assert same == (True, True, True)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- weights that are not finite
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m", [1, 33, 512, 1000])
def test_a_weight_that_is_not_finite_stays_visible(m, dtype):
    n = 9
    W = rnd(1, n, m, dtype=dtype)
    clean = px.Int8Linear(W)
    bad = W.clone()
    for row, v in ((1, float("nan")), (3, float("inf")), (4, -float("inf")), (6, -float("nan"))):
        bad[row, (row * 7) % m] = v
    bad[7, 0], bad[7, m - 1] = float("inf"), float("nan")
    rows = torch.tensor([1, 3, 4, 6, 7])
    lin = px.Int8Linear(bad)
    keep = torch.ones(n, dtype=torch.bool)
    keep[rows] = False
    assert torch.equal(lin.Wq[keep], clean.Wq[keep]) and torch.equal(lin.wscale[keep], clean.wscale[keep])
    assert torch.isnan(lin.wscale[rows]).all() and not lin.Wq[rows].any()
    x = rnd(2, 5, m, dtype=dtype)
    z = lin.forward(x)
    assert torch.isnan(z[:, rows]).all() and torch.equal(z[:, keep], clean.forward(x)[:, keep])
    # the token's quantiser marks the same rows
    q, s = px.quantize_rows(bad)
    assert torch.equal(torch.isnan(s), torch.isnan(lin.wscale)) and not q[rows].any()


@pytest.mark.parametrize("int8_product", [False, True])
def test_a_layer_whose_weight_is_not_finite(int8_product):
    st = state(256, 512, 256, BF, 0)
    st[0][5, 7] = float("nan")
    L = layer(256, 512, 256, BF, (*st[:3], torch.zeros_like(st[3]), torch.zeros_like(st[4])))   # G = I
    L.quantize_weight(int8_product=int8_product)
    z = L.forward(rnd(1, 20, 256, dtype=BF))[0]
    assert torch.isnan(z[:, 5]).all()


def test_the_largest_and_smallest_weights():
    # rows at both ends of the range keep the codes the formula gives
    big, tiny = 3.4028234663852886e38, 2.0 ** -149
    W = torch.tensor([[big, -big, big / 2, 0.0], [127 * tiny, -64 * tiny, 1 * tiny, 0.0], [0.0] * 4], device="cuda")
    lin = px.Int8Linear(W)
    # (the scale is rounded up from big / 127, by 5.6e-8 of it, so big / 2 lies below the border 63.5: 63.499996)
    assert lin.Wq.tolist() == [[127, -127, 63, 0], [127, -64, 1, 0], [0] * 4]
    assert lin.wscale.tolist() == [(W[0, 0] / torch.tensor(127.0, device="cuda")).item(), tiny, 0.0]
