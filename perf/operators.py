"""Cases of the library's 8-bit operators: their inputs, their plain form in
elementary torch operations, the calls a user makes, and the same results in
64 bits.

  product    z = (xs[t] ws[j]) sum_i xq[t][i] Wq[j][i]: int8 tokens by the int8
             weight of a POET-XQ layer, a scale per token and per channel
  gradient   dx of that product from a dz in the layer's dtype: dz[t][j] ws[j]
             quantised row by row, then times Wq over the channels
  norm       h = x + residual, root-mean-square norm of h with a gain, and the
             normalised rows as int8 codes with a scale per row
  norm_grad  dx and dgamma of that norm
  save       an activation kept as int8 codes with a shared power of two per 32
             columns, and read back
  block      the backward of one side of a layer from such a checkpoint X:
             O_j = D_j G_j^T and dG_j = X_j^T D_j for every block j
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
#: Work of the largest listed case, which no drawn case passes.
MOST_FLOPS = 2 * 16384 * 4096 * 14336
MOST_ELEMENTS = 16384 * 14336


def listed():
    return [
        # one sequence generating: a single token through the up-projection of an 8B block
        {"name": "product_T1", "op": "product", "T": 1, "m": 4096, "n": 14336, "dtype": "bf16"},
        # a batch of 48 sequences generating, down-projection
        {"name": "product_T48", "op": "product", "T": 48, "m": 14336, "n": 4096, "dtype": "bf16"},
        # a short ragged prompt through an attention projection, fp32 results
        {"name": "product_T333_fp32", "op": "product", "T": 333, "m": 4096, "n": 1024, "dtype": "fp32"},
        # a whole training batch through the up-projection
        {"name": "product_T16384", "op": "product", "T": 16384, "m": 4096, "n": 14336, "dtype": "bf16"},
        # the backward of the up-projection: contraction over its 14336 channels
        {"name": "gradient_T8192", "op": "gradient", "T": 8192, "m": 4096, "n": 14336, "dtype": "bf16"},
        # a ragged batch at the sizes of a 13B block, no size a multiple of a tile
        {"name": "gradient_T1111_odd", "op": "gradient", "T": 1111, "m": 5120, "n": 13800, "dtype": "bf16"},
        # the norm before a projection: one token, and a whole batch
        {"name": "norm_T1", "op": "norm", "T": 1, "d": 4096, "dtype": "bf16", "residual": True},
        {"name": "norm_T16384", "op": "norm", "T": 16384, "d": 4096, "dtype": "bf16", "residual": True},
        # the norm's backward over a whole batch, with the gradient of the residual stream
        {"name": "norm_grad_T16384", "op": "norm_grad", "T": 16384, "d": 4096, "dtype": "bf16", "residual": True},
        # the P-side activation of an up-projection kept between forward and backward
        {"name": "save_T8192", "op": "save", "T": 8192, "d": 14336, "dtype": "bf16"},
        # the R side of a 4096-wide layer in the backward, from its checkpoint
        {"name": "block_T16384", "op": "block", "T": 16384, "d": 4096, "b": 256, "dtype": "bf16"},
        # a small fp32 layer with ragged tokens
        {"name": "block_T300_fp32", "op": "block", "T": 300, "d": 512, "b": 64, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A feature width: half of the time a multiple of 64, as layers have, else any."""
    w = _log(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.5 else w


def draw(rng):
    op = rng.choice(["product", "product", "gradient", "norm", "norm_grad", "save", "block"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    T = _log(rng, 1, 16384)
    if op in ("product", "gradient"):
        m, n = _width(rng, 64, 14336), _width(rng, 64, 14336)
        T = max(1, min(T, MOST_FLOPS // (2 * m * n)))
        return {"op": op, "T": T, "m": m, "n": n, "dtype": dtype}
    if op == "block":
        b = rng.choice([64, 128, 256, 256, 512]) if dtype == "bf16" else rng.choice([16, 40, 64, 96])
        k = _log(rng, 1, 8192 // b if dtype == "bf16" else 2048 // b)
        return {"op": op, "T": T, "d": b * k, "b": b, "dtype": dtype}
    d = _width(rng, 64, 14336)
    T = max(1, min(T, MOST_ELEMENTS // d))
    case = {"op": op, "T": T, "d": d, "dtype": dtype}
    return case if op == "save" else {**case, "residual": rng.random() < 0.7}


# ---------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", dtype=torch.float32, generator=g)


def _activations(g, T, d, dtype):
    """Tokens as decoder blocks see them: normal, with a few channels many times larger."""
    gain = 1.0 + 15.0 * (torch.rand(d, device="cuda", generator=g) < 0.005)
    return (_normal(g, T, d) * gain).to(DTYPES[dtype])


def _rows_int8(v):
    s = v.abs().amax(1, keepdim=True).clamp_min(1e-30) / 127
    return torch.round(v / s).clamp(-127, 127).to(torch.int8), s[:, 0].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, T, dt = case["op"], case["T"], case["dtype"]
    s = {"case": case}
    if op in ("product", "gradient"):
        m, n = case["m"], case["n"]
        s["Wq"], s["ws"] = _rows_int8(0.02 * _normal(g, n, m))
        if op == "product":
            s["xq"], s["xs"] = _rows_int8(_activations(g, T, m, "fp32"))
        else:
            s["dz"] = _activations(g, T, n, dt)
    elif op in ("norm", "norm_grad"):
        d = case["d"]
        s["gamma"] = 1.0 + 0.1 * _normal(g, d)
        s["x"] = _activations(g, T, d, dt)
        s["r"] = _activations(g, T, d, dt) if case["residual"] else None
        if op == "norm_grad":
            s["dy"] = _normal(g, T, d).to(DTYPES[dt])
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS).float()
    elif op == "save":
        s["x"] = _activations(g, T, case["d"], dt)
    else:
        d, b = case["d"], case["b"]
        s["codes"], s["exps"] = _encode(_activations(g, T, d, "fp32"))
        s["D"] = _normal(g, T, d).to(DTYPES[dt])
        G = torch.eye(b, device="cuda") + 0.05 * _normal(g, d // b, b, b)
        s["G"] = G.to(DTYPES[dt])
    return s


# ---------------------------------------------------------------- plain form
def _quantise(u):
    """Codes and scales of the rows of u (fp32): scale = max|row| / 127 in fp32,
    code = u / scale rounded half to even. The quotient is taken in 64 bits, so
    that a value next to a border falls on its own side of it."""
    top = u.abs().amax(1)
    s = top / torch.full_like(top, 127.0)  # by a tensor: torch turns a division by a number into a product
    q = torch.round(u.double() / s.double()[:, None]).clamp(-127, 127)
    return torch.where(s[:, None] > 0, q, 0.0).float(), s


def _exponent(amax):
    """The smallest e with amax <= 127 * 2^e."""
    f, k = torch.frexp(amax)  # amax = f 2^k, 1/2 <= f < 1
    e = k - 7 + (f * 128 > 127).to(k.dtype)
    return torch.where(amax > 0, e.clamp_min(-126), -126)


def _groups(v):
    T, d = v.shape
    return torch.nn.functional.pad(v, (0, -d % 32)).view(T, -1, 32)


def _encode(v):
    """int8 codes and biased exponents: code = v 2^-e rounded half to even, e shared by 32 columns."""
    T, d = v.shape
    w = _groups(v.float())
    e = _exponent(w.abs().amax(2))
    q = torch.round(torch.ldexp(w, -e[:, :, None]))
    return q.view(T, -1)[:, :d].to(torch.int8).contiguous(), (e + 127).to(torch.uint8)


def _decode(codes, exps):
    T, d = codes.shape
    e = exps.to(torch.int32) - 127
    return torch.ldexp(_groups(codes.float()), e[:, :, None]).view(T, -1)[:, :d]


def _blocks(v, b):
    """[T][d] -> [d/b][T][b]."""
    return v.view(v.shape[0], -1, b).transpose(0, 1)


def _plain(s):
    op, out = s["case"]["op"], DTYPES[s["case"]["dtype"]]
    if op == "product":
        acc = s["xq"].float() @ s["Wq"].float().t()
        return (acc * s["xs"][:, None] * s["ws"]).to(out)
    if op == "gradient":
        q, qs = _quantise(s["dz"].float() * s["ws"])
        return ((q @ s["Wq"].float()) * qs[:, None]).to(out)
    if op == "norm":
        h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(out)
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(1) + EPS)
        q, us = _quantise(hf * s["gamma"])
        scale = rstd * us
        values = (q * scale[:, None]).to(out)
        return (values, scale, rstd) if s["r"] is None else (values, scale, rstd, h)
    if op == "norm_grad":
        h, rstd = s["x"].float(), s["rstd"][:, None]
        p = s["dy"].float() * s["gamma"]
        dx = rstd * (p - h * rstd * rstd * (p * h).mean(1, keepdim=True))
        if s["r"] is not None:
            dx = dx + s["r"].float()
        return dx.to(out), (s["dy"].float() * (h * rstd)).sum(0)
    if op == "save":
        codes, exps = _encode(s["x"])
        return _decode(codes, exps).to(out)
    b, D = s["case"]["b"], s["D"].float()
    X = _decode(s["codes"], s["exps"])
    O = _blocks(D, b) @ s["G"].float().transpose(1, 2)
    dG = _blocks(X, b).transpose(1, 2) @ _blocks(D, b)
    return O.transpose(0, 1).reshape(D.shape).to(out), dG


def _own(s):
    import orthogonal_equivalence_b200 as px
    op, out = s["case"]["op"], DTYPES[s["case"]["dtype"]]
    if op == "product":
        return px.matmul_int8(s["xq"], s["xs"], s["Wq"], s["ws"], out)
    if op == "gradient":
        return px.matmul_int8_grad(s["dz"], s["Wq"], s["ws"])
    if op == "norm":
        r = px.rmsnorm_quantize(s["x"], s["gamma"], s["r"], EPS)
        values = px.dequantize_rows(r.codes, r.scale, out)
        return (values, r.scale, r.rstd) if s["r"] is None else (values, r.scale, r.rstd, r.h)
    if op == "norm_grad":
        return px.rmsnorm_backward(s["dy"], s["x"], s["gamma"], s["rstd"], s["r"])
    if op == "save":
        return px.checkpoint_load(px.checkpoint_save(s["x"]), out)
    return px.block_backward(px.Checkpoint(s["codes"], s["exps"]), s["D"], s["G"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- work
def work(case):
    op, T, es = case["op"], case["T"], SIZE[case["dtype"]]
    if op in ("product", "gradient"):
        m, n = case["m"], case["n"]
        io = T * m + 4 * T + T * n * es if op == "product" else T * n * es + T * m * es
        return {"bytes": io + n * m + 4 * n, "flops": 2 * T * n * m}
    d = case["d"]
    if op == "norm":
        return {"bytes": T * d * es * (4 if case["residual"] else 2) + 4 * d + 8 * T, "flops": 6 * T * d}
    if op == "norm_grad":
        return {"bytes": T * d * es * (4 if case["residual"] else 3) + 8 * d + 4 * T, "flops": 10 * T * d}
    if op == "save":
        return {"bytes": T * d * es * 2, "flops": 4 * T * d}
    b = case["b"]
    held = T * d + T * ((d + 31) // 32)
    return {"bytes": held + 2 * T * d * es + d * b * es + 4 * d * b, "flops": 4 * T * d * b}


# ---------------------------------------------------------------- in 64 bits
def _codes64(u):
    """Rows of fp32 values -> (codes, scales) as fp64, from the quantiser's definition."""
    top = u.abs().max(dim=1).values
    s = top.div(torch.full_like(top, 127.0)).double()
    live = s > 0
    q = u.double().div(torch.where(live, s, 1.0).unsqueeze(1)).round()
    return q.clamp(-127.0, 127.0) * live.unsqueeze(1), s


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        z = torch.mm(s["xq"].double(), s["Wq"].double().T)
        return z.mul_(s["xs"].double().unsqueeze(1)).mul_(s["ws"].double())
    if op == "gradient":
        q, qs = _codes64(torch.mul(s["dz"].float(), s["ws"]))
        return torch.mm(q, s["Wq"].double()).mul_(qs.unsqueeze(1))
    if op == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            # the residual stream is held in the layer's dtype: that rounding belongs to the operator
            h = (s["x"].float() + s["r"].float()).to(DTYPES[case["dtype"]]).double()
        rstd = (h.pow(2).sum(1) / case["d"] + EPS).pow(-0.5)
        q, us = _codes64(torch.mul(h.float(), s["gamma"]))
        scale = us * rstd
        got = (q * scale.unsqueeze(1), scale, rstd)
        return got if s["r"] is None else got + (s["x"].double() + s["r"].double(),)
    if op == "norm_grad":
        x, dy, w, rs = s["x"].double(), s["dy"].double(), s["gamma"].double(), s["rstd"].double()
        xn = x * rs.unsqueeze(1)
        t = dy * w
        dx = (t - xn * (t * xn).sum(1, keepdim=True) / case["d"]) * rs.unsqueeze(1)
        if s["r"] is not None:
            dx += s["r"].double()
        return dx, torch.einsum("td,td->d", dy, xn)
    if op == "save":
        x = s["x"].double()
        T, d = x.shape
        w = torch.cat([x, x.new_zeros(T, -d % 32)], 1).reshape(T, -1, 32)
        top = w.abs().amax(2, keepdim=True)
        e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -119) / 127))
        e = torch.where(top > 127 * torch.exp2(e), e + 1, e)  # log2 may round across a whole number
        e = torch.where(top <= 127 * torch.exp2(e - 1), e - 1, e).clamp_min(-126)
        return ((w / torch.exp2(e)).round() * torch.exp2(e)).reshape(T, -1)[:, :d]
    T, d, b = case["T"], case["d"], case["b"]
    power = torch.exp2(s["exps"].double() - 127).repeat_interleave(32, dim=1)[:, :d]
    X = (s["codes"].double() * power).reshape(T, d // b, b)
    D = s["D"].double().reshape(T, d // b, b)
    O = torch.einsum("tjc,jrc->tjr", D, s["G"].double()).reshape(T, d)
    return O, torch.einsum("tjr,tjc->jrc", X, D)
