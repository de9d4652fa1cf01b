"""Layer norm, linear layers and products grouped by expert, with their
gradients, against the formulas in 64 bits.

Tolerances count roundings, element by element.  u = eps/2 of the output's
type is the store's rounding.  A sum of n products in fp32 is off by at most
n 2^-23 sum|a b| (2^-23 and not 2^-24: the matrix instruction may truncate).
Where the kernel rounds an operand first (g = dy act'(pre) of the linear
layer's gradient), that adds u sum|a b|.  fp32 elementary functions are taken
as good to 2^-18 of their argument's scale (a fast exponential of an argument
up to 2^5 is off by at most 2^5 2^-23 relative).
"""
import math

import pytest
import torch

import expert_ffn_dispatch_amd as moe

pytestmark = pytest.mark.gpu

DEV = "cuda"
ACC = 2.0 ** -23
FUN = 2.0 ** -18
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def u(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Absolute rounding of values below the type's normal range."""
    return torch.finfo(t).tiny * torch.finfo(t).eps


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def strided(t, pad, shift=0):
    """The same values with `pad` more elements to a row and `shift` elements in front."""
    r, c = t.shape
    buf = torch.full((r * (c + pad) + shift,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[shift:].view(r, c + pad)[:, :c]
    v.copy_(t)
    return v


def check(got, ref, tol, what):
    assert tuple(got.shape) == tuple(ref.shape), what
    d = (got.double() - ref).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at "
                           f"{[int(i) for i in bad.nonzero()[0]]}: got {got[tuple(bad.nonzero()[0])].item()}, "
                           f"want {ref[tuple(bad.nonzero()[0])].item()}, worst ratio {(d / tol).nan_to_num(1e30).max().item():.2f}")


# ------------------------------------------------------------------- norm

def norm_ref(x, gamma, beta, eps, rms):
    x = x.double()
    mu = torch.zeros(x.shape[0], 1, dtype=torch.float64, device=x.device) if rms else x.mean(1, keepdim=True)
    rstd = 1 / ((x - mu).pow(2).mean(1, keepdim=True) + eps).sqrt()
    n = (x - mu) * rstd
    g = 1.0 if gamma is None else gamma.double()
    b = 0.0 if beta is None else beta.double()
    return n * g + b, mu[:, 0], rstd[:, 0], n


NORM_SHAPES = [(1, 1), (1, 2048), (3, 7), (2, 64), (5, 63), (1, 16384), (4, 513), (7, 1111), (1500, 256), (1030, 2048),
               (1025, 4096), (33, 5120), (6, 8200), (5, 4097), (3, 16383)]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype,pt", [(BF, BF), (BF, F32), (HF, HF), (F32, F32)])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm_forward(rows, cols, dtype, pt, rms):
    g = gen(rows * 31 + cols)
    x = (torch.randn(rows, cols, generator=g, device=DEV) * 2 + 5).to(dtype)   # a mean well above the deviation
    gamma, beta = randn(g, cols, dtype=pt), randn(g, cols, dtype=pt)
    y, mean, rstd = moe.moe_layer_norm(x, gamma, beta, eps=1e-5, rms=rms, want_stats=True)
    ref, mu, rs, n = norm_ref(x, gamma, beta, 1e-5, rms)
    # fp32 statistics: mu off by cols-independent tree sums, at most 2^-18 of max|x| (16 sums in a thread, 10 levels)
    scale = x.double().abs().max(1).values
    check(mean, mu, FUN * scale + 1e-30, "mean")
    check(rstd, rs, FUN * rs * (1 + scale * rs), "rstd")
    err = FUN * (1 + (scale * rs)[:, None]) * (n.abs() + 1) * gamma.double().abs() + 2 * ACC * beta.double().abs()
    check(y, ref, u(dtype) * ref.abs() + 1.01 * err + tiny(dtype), "y")


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype,pt", [(BF, BF), (BF, F32), (HF, HF), (F32, F32)])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm_backward(rows, cols, dtype, pt, rms):
    g = gen(rows * 37 + cols)
    x = (torch.randn(rows, cols, generator=g, device=DEV) + 0.5).to(dtype)
    gamma = randn(g, cols, dtype=pt)
    dy = randn(g, rows, cols, dtype=dtype)
    _, mu, rs, _ = norm_ref(x, gamma, None, 1e-5, rms)
    mean, rstd = mu.float(), rs.float()
    dx, dgamma, dbeta = moe.moe_layer_norm_backward(dy, x, gamma, None if rms else mean, rstd, rms=rms)
    mu, rs = mean.double()[:, None], rstd.double()[:, None]
    n = (x.double() - mu) * rs
    gg = dy.double() * gamma.double()
    m1 = 0 if rms else gg.mean(1, keepdim=True)
    m2 = (gg * n).mean(1, keepdim=True)
    ref = rs * (gg - m1 - n * m2)
    # each fp32 term is off by a few 2^-24 of its size, the means by 2^-18 of the mean of |terms|
    en = 4 * ACC * ((x.double().abs() + mu.abs()) * rs)
    terms = gg.abs() + gg.abs().mean(1, keepdim=True) + n.abs() * (gg * n).abs().mean(1, keepdim=True)
    err = rs * (FUN * terms + en * (m2.abs() + gg.abs().mean(1, keepdim=True)))
    check(dx, ref, u(dtype) * ref.abs() + err + tiny(dtype), "dx")
    acc = (rows + 64) * ACC
    rg = (dy.double() * n).sum(0)
    check(dgamma, rg, u(pt) * rg.abs() + acc * (dy.double() * n).abs().sum(0) + (dy.double().abs() * en).sum(0) + tiny(pt), "dgamma")
    rb = dy.double().sum(0)
    check(dbeta, rb, u(pt) * rb.abs() + acc * dy.double().abs().sum(0) + tiny(pt), "dbeta")


def test_norm_gradient_against_differences():
    """dx, dgamma, dbeta of a scalar loss against central differences of the fp32 forward's formula in 64 bits."""
    g = gen(3)
    rows, cols = 4, 24
    x, gamma, beta = (torch.randn(s, generator=g, device=DEV) for s in ((rows, cols), (cols,), (cols,)))
    dy = torch.randn(rows, cols, generator=g, device=DEV)
    y, mean, rstd = moe.moe_layer_norm(x, gamma, beta, want_stats=True)
    dx, dgamma, dbeta = moe.moe_layer_norm_backward(dy, x, gamma, mean, rstd)
    h = 1e-4

    def loss(a, b, c):
        return (norm_ref(a, b, c, 1e-5, False)[0] * dy.double()).sum()

    args = [t.double() for t in (x, gamma, beta)]
    for k, got in enumerate((dx, dgamma, dbeta)):
        for i in range(0, args[k].numel(), 5):
            lo, hi = [t.clone() for t in args], [t.clone() for t in args]
            lo[k].view(-1)[i] -= h
            hi[k].view(-1)[i] += h
            diff = (loss(*hi) - loss(*lo)) / (2 * h)
            # third derivatives of order 1e2 times h^2 / 6, and the fp32 result
            assert abs(got.view(-1)[i].item() - diff.item()) < 2e-5 * (1 + abs(diff.item()))


@pytest.mark.parametrize("cols,pad,shift", [(64, 8, 0), (64, 3, 0), (96, 8, 1), (1024, 24, 8), (33, 1, 2)])
def test_norm_strides(cols, pad, shift):
    g = gen(cols)
    x, gamma, dy = randn(g, 9, cols), randn(g, cols), randn(g, 9, cols)
    want = moe.moe_layer_norm(x, gamma, want_stats=True)
    xs, out = strided(x, pad, shift), strided(torch.zeros_like(x), pad, shift)
    y, mean, rstd = moe.moe_layer_norm(xs, gamma, want_stats=True, y=out)
    # another load path may sum in another order: one rounding step
    check(y, want[0].double(), 2 * u(BF) * want[0].double().abs() + 1e-6, "y")
    base = out._base if out._base is not None else out
    pads = base.reshape(-1)[shift:].view(9, cols + pad)[:, cols:]
    assert torch.isnan(pads).all(), "the space between rows was written"
    a = moe.moe_layer_norm_backward(dy, x, gamma, mean, rstd)
    b = moe.moe_layer_norm_backward(strided(dy, pad, shift), xs, gamma, mean, rstd)
    for p, q in zip(a, b):
        check(q, p.double(), 2 * u(BF) * p.double().abs() + 1e-5, "gradient")


def test_norm_many_rows():
    """More rows than one launch takes."""
    g = gen(12)
    x = randn(g, 2 ** 21 + 5, 8)
    y, mean, rstd = moe.moe_layer_norm(x, want_stats=True)
    ref, mu, rs, n = norm_ref(x, None, None, 1e-5, False)
    scale = x.double().abs().max(1).values
    check(mean, mu, FUN * scale + 1e-30, "mean")
    check(y, ref, u(BF) * ref.abs() + FUN * (1 + (scale * rs)[:, None]) * (n.abs() + 1), "y")


def test_norm_in_place_and_empty():
    g = gen(1)
    x = randn(g, 300, 640)
    want = moe.moe_layer_norm(x)
    y = x.clone()
    assert torch.equal(moe.moe_layer_norm(y, y=y), want)
    e = torch.empty(0, 640, dtype=BF, device=DEV)
    assert moe.moe_layer_norm(e).shape == (0, 640)
    z = torch.empty(0, dtype=F32, device=DEV)
    dx, dg, db = moe.moe_layer_norm_backward(e, e, None, z, z)
    assert dx.shape == (0, 640) and not dg.any() and not db.any()
    # a row of equal values: n = 0, dx finite
    c = torch.full((2, 640), 3.0, dtype=BF, device=DEV)
    y, m, r = moe.moe_layer_norm(c, want_stats=True)
    assert not y.any() and torch.isfinite(r).all()
    # NaN and infinity stay in their rows
    x[7, 3] = float("nan")
    x[9, 5] = float("inf")
    y = moe.moe_layer_norm(x)
    ok = torch.ones(300, dtype=torch.bool, device=DEV)
    ok[7] = ok[9] = False
    assert torch.equal(y[ok], want[ok]) and torch.isnan(y[7]).all()


# --------------------------------------------------------------- products

def act_ref(z, act):
    return {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "gelu": lambda v: v * torch.special.ndtr(v),
            "gelu_tanh": lambda v: 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))),
            "silu": lambda v: v * torch.sigmoid(v)}[act](z)


def act_grad_ref(z, act):
    z = z.detach().clone().requires_grad_()
    act_ref(z, act).sum().backward()
    return torch.where(z == 0, torch.zeros_like(z), z.grad) if act == "relu" else z.grad


ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
# rows, in, out: one token, ragged tiles, odd widths, several tiles, contraction slices
LIN_SHAPES = [(1, 64, 64), (1, 2048, 512), (3, 1, 1), (2, 7, 5), (17, 72, 40), (37, 512, 256), (64, 1000, 136),
              (130, 264, 392), (129, 65, 131), (300, 4096, 64), (257, 768, 512), (1, 4097, 33), (700, 1001, 1003), (333, 1003, 96),
              (40, 1536, 6200), (33, 256, 12400)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,n_in,n_out", LIN_SHAPES)
def test_linear_forward(rows, n_in, n_out, act):
    g = gen(rows + n_in + n_out)
    dtype = HF if (rows + n_out) % 2 else BF
    x, w = randn(g, rows, n_in, dtype=dtype), randn(g, n_out, n_in, dtype=dtype, scale=n_in ** -0.5)
    bias = randn(g, n_out, dtype=F32 if act in ("relu", "silu") else dtype)
    res = randn(g, rows, n_out, dtype=dtype) if act != "gelu" else None
    y, pre = moe.moe_linear(x, w, bias, res, act=act, want_pre=True)
    z = x.double() @ w.double().T + bias.double()
    ez = (n_in + 2) * ACC * (x.double().abs() @ w.double().abs().T + bias.double().abs())
    check(pre, z, u(dtype) * z.abs() + 1.01 * ez + tiny(dtype), "pre")
    ref = act_ref(z, act)
    r = 0 if res is None else res.double()
    # slopes of the activations are at most 1.13
    err = 1.2 * ez + FUN * ref.abs() + ACC * z.abs()
    check(y, ref + r, u(dtype) * (ref + r).abs() + 1.01 * err + 2 * ACC * (ref + r).abs() + tiny(dtype), "y")
    # the same without what is optional
    y2 = moe.moe_linear(x, w, act=act)
    z2 = x.double() @ w.double().T
    ref2 = act_ref(z2, act)
    check(y2, ref2, u(dtype) * ref2.abs() + 1.01 * (1.2 * ez + FUN * ref2.abs() + ACC * z2.abs()) + tiny(dtype), "y, plain")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,n_in,n_out", LIN_SHAPES + [(2100, 128, 72)])
def test_linear_backward(rows, n_in, n_out, act):
    g = gen(rows + n_in + 3 * n_out)
    dtype = BF if (rows + n_out) % 2 else HF
    bt = F32 if act in ("none", "gelu") else dtype
    x, w = randn(g, rows, n_in, dtype=dtype), randn(g, n_out, n_in, dtype=dtype, scale=n_in ** -0.5)
    dy, pre = randn(g, rows, n_out, dtype=dtype), randn(g, rows, n_out, dtype=dtype, scale=2.0)
    dx, dw, db = moe.moe_linear_backward(dy, x, w, None if act == "none" else pre, act=act, want_dbias=True,
                                         bias_dtype=bt, dw_dtype=F32 if act == "relu" else None)
    G = dy.double() * (1 if act == "none" else act_grad_ref(pre.double(), act))
    eg = (0 if act in ("none", "relu") else u(dtype)) * G.abs() + (0 if act in ("none", "relu") else FUN) * dy.double().abs() \
        + tiny(dtype)
    W, X = w.double(), x.double()
    ref = G @ W
    check(dx, ref, u(dtype) * ref.abs() + 1.01 * (eg + n_out * ACC * G.abs()) @ W.abs() + tiny(dtype), "dx")
    ref = G.T @ X
    ut = u(dw.dtype)
    check(dw, ref, ut * ref.abs() + 1.01 * (eg + rows * ACC * G.abs()).T @ X.abs() + tiny(dw.dtype), "dw")
    ref = G.sum(0)
    es = (0 if act in ("none", "relu") else FUN) * dy.double().abs() + (rows + 8) * ACC * G.abs()
    check(db, ref, u(bt) * ref.abs() + 1.01 * es.sum(0) + tiny(bt), "dbias")


def test_linear_gradient_against_differences():
    g = gen(11)
    x, w, b = randn(g, 6, 24), randn(g, 16, 24, scale=0.2), randn(g, 16, dtype=F32)
    dy = randn(g, 6, 16)
    for act in ACTS[1:]:
        z = x.double() @ w.double().T + b.double()
        pre = z.to(BF)
        dx, dw, db = moe.moe_linear_backward(dy, x, w, pre, act=act, want_dbias=True, bias_dtype=F32)
        h = 1e-5
        G = dy.double() * (act_ref(pre.double() + h, act) - act_ref(pre.double() - h, act)) / (2 * h)
        if act == "relu":
            G = dy.double() * (pre > 0)
        eg = u(BF) * G.abs() + 1e-5 * dy.double().abs()
        check(dx, G @ w.double(), u(BF) * (G @ w.double()).abs() + 1.01 * eg @ w.double().abs() + 1e-6, "dx " + act)
        check(dw, G.T @ x.double(), u(BF) * (G.T @ x.double()).abs() + 1.01 * eg.T @ x.double().abs() + 1e-6, "dw " + act)
        check(db, G.sum(0), 1e-4 * (1 + dy.double().abs().sum(0)), "dbias " + act)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", ACTS[1:])
def test_linear_activation_at_large_values(act, dtype):
    """Far out an activation is z or 0 and its slope 1 or 0, exactly; NaN stays NaN."""
    top = float(torch.finfo(dtype).max)
    z = torch.tensor([129.0, 300.0, 1e4, 6e4, min(1e20, top), top, top / 3, 200.0], device=DEV).to(dtype)
    z = torch.stack([z, -z])
    eye = torch.eye(8, dtype=dtype, device=DEV)
    y, pre = moe.moe_linear(z, eye, act=act, want_pre=True)
    assert torch.equal(pre, z) and torch.equal(y, z.clamp(min=0))
    pre = torch.cat([z, torch.full_like(z[:1], float("inf")), torch.full_like(z[:1], float("-inf"))])
    dx, dw, db = moe.moe_linear_backward(torch.ones_like(pre), pre.clamp(-1, 1), eye, pre, act=act, want_dbias=True,
                                         bias_dtype=F32)
    slope = (pre > 0).to(dtype)
    assert torch.equal(dx, slope) and torch.equal(db, slope.float().sum(0))
    assert torch.equal(dw, torch.full_like(eye, 2.0))     # two rows of slope 1 and x = 1
    pre[1, 3] = float("nan")
    dx = moe.moe_linear_backward(torch.ones_like(pre), pre.clamp(-1, 1), eye, pre, act=act)[0]
    if act != "relu":                             # whose slope is that of z > 0
        assert torch.isnan(dx[1, 3])
    assert torch.equal(dx[0], slope[0])


@pytest.mark.parametrize("n_in,n_out,pad,shift", [(128, 192, 8, 0), (128, 192, 3, 0), (136, 72, 16, 8), (96, 64, 8, 1),
                                                  (77, 51, 2, 3)])
def test_linear_strides(n_in, n_out, pad, shift):
    g = gen(n_in)
    x, w, r, dy = randn(g, 70, n_in), randn(g, n_out, n_in, scale=0.1), randn(g, 70, n_out), randn(g, 70, n_out)
    y0, p0 = moe.moe_linear(x, w, None, r, act="silu", want_pre=True)
    S = lambda t: strided(t, pad, shift)  # noqa: E731
    out, pre = S(torch.zeros_like(y0)), S(torch.zeros_like(y0))
    moe.moe_linear(S(x), S(w), None, S(r), act="silu", y=out, pre=pre)
    # another order of the same fp32 sums: one rounding step of the stored values
    check(out, y0.double(), 2 * u(BF) * y0.double().abs() + 1e-5, "y")
    check(pre, p0.double(), 2 * u(BF) * p0.double().abs() + 1e-5, "pre")
    for t in (out, pre):
        pads = t._base.reshape(-1)[shift:].view(70, n_out + pad)[:, n_out:]
        assert torch.isnan(pads).all(), "the space between rows was written"
    a = moe.moe_linear_backward(dy, x, w, p0, act="silu", want_dbias=True)
    b = moe.moe_linear_backward(S(dy), S(x), S(w), S(p0), act="silu", want_dbias=True)
    for p, q in zip(a, b):
        check(q, p.double(), 2 * u(BF) * p.double().abs() + 1e-4, "gradient")


@pytest.mark.parametrize("rows", [1, 20, 64])
def test_linear_few_rows_misaligned(rows):
    """Shapes for the kernel of a few rows whose pointers do not suit it."""
    g = gen(rows)
    x, w = randn(g, rows, 256), randn(g, 96, 256, scale=0.06)
    ref = x.double() @ w.double().T
    tol = u(BF) * ref.abs() + 1.01 * 256 * ACC * x.double().abs() @ w.double().abs().T + tiny(BF)
    check(moe.moe_linear(x, w), ref, tol, "aligned")
    check(moe.moe_linear(strided(x, 8, 1), w), ref, tol, "x")
    check(moe.moe_linear(x, strided(w, 8, 3)), ref, tol, "w")
    check(moe.moe_linear(strided(x, 3, 1), strided(w, 5, 2)), ref, tol, "both")


@pytest.mark.parametrize("rows,n_in,n_out", [(4400, 1024, 4400), (2200, 512, 4000), (4001, 520, 4361)])
def test_linear_rounds_with_a_cut_tail(rows, n_in, n_out):
    """More tiles than the card has CUs, the last round of them cut along the contraction."""
    g = gen(rows)
    x, w, b = randn(g, rows, n_in), randn(g, n_out, n_in, scale=n_in ** -0.5), randn(g, n_out)
    X, W = x.double(), w.double()
    ref = X @ W.T + b.double()
    check(moe.moe_linear(x, w, b), ref, u(BF) * ref.abs() + 1.01 * (n_in + 2) * ACC * (X.abs() @ W.abs().T + b.double().abs())
          + tiny(BF), "y")
    dy = randn(g, rows, n_out)
    dx, dw, db = moe.moe_linear_backward(dy, x, w, want_dbias=True, dw_dtype=F32)
    D = dy.double()
    check(dx, D @ W, u(BF) * (D @ W).abs() + 1.01 * n_out * ACC * D.abs() @ W.abs() + tiny(BF), "dx")
    check(dw, D.T @ X, u(F32) * (D.T @ X).abs() + rows * ACC * D.abs().T @ X.abs(), "dw")
    check(db, D.sum(0), u(BF) * D.sum(0).abs() + (rows + 8) * ACC * D.abs().sum(0) + tiny(BF), "dbias")


def test_linear_residual_in_place_and_empty():
    g = gen(5)
    x, w, r = randn(g, 50, 64), randn(g, 80, 64), randn(g, 50, 80)
    want = moe.moe_linear(x, w, None, r)
    y = r.clone()
    assert torch.equal(moe.moe_linear(x, w, None, y, y=y), want)
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    assert moe.moe_linear(e, w).shape == (0, 80)
    dx, dw, db = moe.moe_linear_backward(torch.empty(0, 80, dtype=BF, device=DEV), e, w, want_dbias=True)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    # NaN stays in its row (forward) and column (weights)
    x[3, 1] = float("nan")
    y = moe.moe_linear(x, w, None, r)
    ok = torch.arange(50, device=DEV) != 3
    assert torch.equal(y[ok], want[ok]) and torch.isnan(y[3]).all()


def offsets_of(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device=DEV)


GROUPS = [
    ([5], 64, 64), ([1], 1, 1), ([0], 40, 24), ([0, 0, 3, 0], 72, 136), ([1] * 7, 128, 256), ([130, 0, 1, 33, 257], 192, 264),
    ([31, 32, 33, 0, 64, 65, 127, 128, 129], 256, 128), ([3, 9, 0, 2], 65, 131), ([700, 0, 2, 600], 512, 320),
    ([2] * 256, 64, 72), ([300, 0, 77], 2048, 2048), ([120, 200], 2056, 1999), ([0] * 100 + [50] + [0] * 59, 128, 128), ([20] * 16, 1024, 768),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,n_in,n_out", GROUPS, ids=[f"{len(c)}x{sum(c)}-{i}-{o}" for c, i, o in GROUPS])
def test_grouped(counts, n_in, n_out, dtype):
    g = gen(sum(counts) + n_in)
    front, back = 3, 5                              # rows outside every group
    E, rows = len(counts), sum(counts) + front + back
    off = offsets_of(counts, front)
    x, dy = randn(g, rows, n_in, dtype=dtype), randn(g, rows, n_out, dtype=dtype)
    w = randn(g, E, n_out, n_in, dtype=dtype, scale=n_in ** -0.5)
    for t in (x, dy):
        t[:front] = float("nan")
        t[rows - back:] = float("nan")
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = float("nan")                     # never read
    y = torch.full((rows, n_out), 7.0, dtype=dtype, device=DEV)
    dx = torch.full((rows, n_in), 7.0, dtype=dtype, device=DEV)
    moe.moe_grouped_matmul(x, off, w, y=y)
    moe.moe_grouped_matmul_dgrad(dy, off, w, dx=dx)
    dw = moe.moe_grouped_matmul_wgrad(dy, x, off)
    dwf = moe.moe_grouped_matmul_wgrad(dy, x, off, dtype=F32)
    for t in (y, dx):
        assert (t[:front] == 7).all() and (t[rows - back:] == 7).all(), "rows outside the groups were written"
    b = front
    for e, c in enumerate(counts):
        X, D, W = x[b:b + c].double(), dy[b:b + c].double(), w[e].double()
        if c:
            ref = X @ W.T
            check(y[b:b + c], ref, u(dtype) * ref.abs() + 1.01 * n_in * ACC * X.abs() @ W.abs().T + tiny(dtype), f"y {e}")
            ref = D @ W
            check(dx[b:b + c], ref, u(dtype) * ref.abs() + 1.01 * n_out * ACC * D.abs() @ W.abs() + tiny(dtype), f"dx {e}")
        ref = D.T @ X
        acc = (c + 1) * ACC * D.abs().T @ X.abs()
        check(dw[e], ref, u(dtype) * ref.abs() + 1.01 * acc + tiny(dtype), f"dw {e}")
        check(dwf[e], ref, u(F32) * ref.abs() + acc + 1e-30, f"dw fp32 {e}")
        b += c


def test_grouped_strides_and_empty():
    g = gen(2)
    off = offsets_of([10, 0, 21])
    for n_in, n_out, pad, shift in ((64, 72, 8, 0), (64, 72, 1, 0), (40, 56, 8, 4)):
        x, dy, w = randn(g, 31, n_in), randn(g, 31, n_out), randn(g, 3, n_out, n_in)
        S = lambda t: strided(t, pad, shift)  # noqa: E731
        y, dx = S(torch.zeros_like(dy)), S(torch.zeros_like(x))
        moe.moe_grouped_matmul(S(x), off, w, y=y)
        moe.moe_grouped_matmul_dgrad(S(dy), off, w, dx=dx)
        a = moe.moe_grouped_matmul(x, off, w), moe.moe_grouped_matmul_dgrad(dy, off, w), moe.moe_grouped_matmul_wgrad(dy, x, off)
        for p, q in zip(a, (y, dx, moe.moe_grouped_matmul_wgrad(S(dy), S(x), off))):
            # another order of the same fp32 sums (terms up to ~10): one rounding step
            check(q, p.double(), 2 * u(BF) * p.double().abs() + 1e-4, "strided")
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    zero = torch.zeros(4, dtype=torch.int32, device=DEV)
    w = randn(g, 3, 72, 64)
    assert moe.moe_grouped_matmul(e, zero, w).shape == (0, 72)
    assert moe.moe_grouped_matmul_dgrad(torch.empty(0, 72, dtype=BF, device=DEV), zero, w).shape == (0, 64)
    assert not moe.moe_grouped_matmul_wgrad(torch.empty(0, 72, dtype=BF, device=DEV), e, zero).any()


def test_grouped_offsets_are_clamped():
    """Offsets past the rows, below zero or decreasing count as the nearest valid ones: no access leaves the buffers."""
    g = gen(8)
    x, dy, w = randn(g, 40, 64), randn(g, 40, 72), randn(g, 3, 72, 64)
    bad = torch.tensor([-5, 10, 7, 1000], dtype=torch.int32, device=DEV)
    good = ((0, 10, 0), (7, 40, 2))
    y = moe.moe_grouped_matmul(x, bad, w)
    assert torch.equal(y[:7], moe.moe_grouped_matmul(x[:10], offsets_of([10, 0, 0]), w)[:7])
    assert torch.equal(y[10:], moe.moe_grouped_matmul(x[7:], offsets_of([0, 0, 33]), w)[3:])
    dw = moe.moe_grouped_matmul_wgrad(dy, x, bad, dtype=F32)
    for lo, hi, e in good:
        ref = dy[lo:hi].double().T @ x[lo:hi].double()
        check(dw[e], ref, 64 * ACC * dy[lo:hi].double().abs().T @ x[lo:hi].double().abs() + 1e-30, f"dw {e}")
    assert not dw[1].any()


# ------------------------------------------------- together, streams, graphs

def test_dense_block_step():
    """A pre-norm feed-forward block, x + W2 gelu(W1 norm(x) + b1) + b2, forward
    and backward through the operators, against the same in 64 bits with the
    operators' roundings bounded by the chain's condition (relative 2-norm: six
    bf16 roundings of 2^-9 each way, so 2% is a factor of two above their sum)."""
    g = gen(21)
    R, M, H = 333, 256, 512
    x = randn(g, R, M)
    ga, be = randn(g, M, scale=0.2) + 1, randn(g, M, scale=0.1)
    w1, b1 = randn(g, H, M, scale=M ** -0.5), randn(g, H, scale=0.1)
    w2, b2 = randn(g, M, H, scale=H ** -0.5), randn(g, M, scale=0.1)
    dout = randn(g, R, M)
    n, mean, rstd = moe.moe_layer_norm(x, ga, be, want_stats=True)
    h, pre = moe.moe_linear(n, w1, b1, act="gelu", want_pre=True)
    out = moe.moe_linear(h, w2, b2, residual=x)
    dh, dw2, db2 = moe.moe_linear_backward(dout, h, w2, want_dbias=True)
    dn, dw1, db1 = moe.moe_linear_backward(dh, n, w1, pre, act="gelu", want_dbias=True)
    dx, dga, dbe = moe.moe_layer_norm_backward(dn, x, ga, mean, rstd)
    dx = dx.double() + dout.double()
    leaves = [t.double().requires_grad_() for t in (x, ga, be, w1, b1, w2, b2)]
    X, GA, BE, W1, B1, W2, B2 = leaves
    mu = X.mean(1, keepdim=True)
    N = (X - mu) / ((X - mu).pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * GA + BE
    O = act_ref(N @ W1.T + B1, "gelu") @ W2.T + B2 + X
    O.backward(dout.double())
    for name, got, ref in [("out", out, O.detach())] + [(k, v, t.grad) for k, v, t in zip(
            ("dx", "dgamma", "dbeta", "dw1", "db1", "dw2", "db2"), (dx, dga, dbe, dw1, db1, dw2, db2), leaves)]:
        rel = ((got.double() - ref).norm() / ref.norm()).item()
        assert rel < 2e-2, (name, rel)


def test_expert_step_with_dispatch():
    """Norm -> route -> permute -> grouped products with a SwiGLU between ->
    combine, and the experts' gradients back to the tokens (moe_combine of the
    rows' gradients with weight one adds a token's rows), against 64 bits."""
    g = gen(33)
    N, M, E, k, H = 200, 256, 8, 2, 128
    d = moe.dims(N, M, E, k, H)
    x = randn(g, N, M)
    xn, mean, rstd = moe.moe_layer_norm(x, randn(g, M, scale=0.1) + 1, want_stats=True, rms=True)
    wr = randn(g, M, E, scale=M ** -0.5)
    ids, wts = moe.moe_route(d, xn, wr)
    perm = moe.moe_permute(d, ids, x=xn, want_x_sorted=True)
    xs, off, a2s, s2a = perm["x_sorted"], perm["expert_offsets"], perm["assign_to_sorted"], perm["sorted_to_assign"]
    wg, wu = randn(g, E, H, M, scale=M ** -0.5), randn(g, E, H, M, scale=M ** -0.5)
    wd = randn(g, E, M, H, scale=H ** -0.5)
    gt, up = moe.moe_grouped_matmul(xs, off, wg), moe.moe_grouped_matmul(xs, off, wu)
    hid = (torch.nn.functional.silu(gt.float()) * up.float()).to(BF)
    y = moe.moe_grouped_matmul(hid, off, wd)
    out = moe.moe_combine(d, y, a2s, wts)
    # against the framework's fused layer on the same rows
    fused = moe.moe_grouped_ffn(d, xs, off, wg, wu, wd)
    assert ((y.float() - fused.float()).norm() / fused.float().norm()).item() < 1e-2
    dout = randn(g, N, M)
    rw = wts.view(-1)[s2a.long()]
    dy = (dout[(s2a // k).long()].float() * rw[:, None]).to(BF)
    dh = moe.moe_grouped_matmul_dgrad(dy, off, wd)
    dwd = moe.moe_grouped_matmul_wgrad(dy, hid, off, dtype=F32)
    s = torch.sigmoid(gt.float())
    dg = (dh.float() * up.float() * s * (1 + gt.float() * (1 - s))).to(BF)
    du = (dh.float() * gt.float() * s).to(BF)
    dwg, dwu = moe.moe_grouped_matmul_wgrad(dg, xs, off, dtype=F32), moe.moe_grouped_matmul_wgrad(du, xs, off, dtype=F32)
    dxs = (moe.moe_grouped_matmul_dgrad(dg, off, wg).float() + moe.moe_grouped_matmul_dgrad(du, off, wu).float()).to(BF)
    dxn = moe.moe_combine(d, dxs, a2s)
    leaves = [t.double().requires_grad_() for t in (xn, wg, wu, wd)]
    X, WG, WU, WD = leaves
    O = torch.zeros(N, M, dtype=torch.float64, device=DEV)
    for e in range(E):
        for j in range(k):
            t = (ids[:, j] == e).nonzero()[:, 0]
            a = torch.nn.functional.silu(X[t] @ WG[e].T) * (X[t] @ WU[e].T)
            O = O.index_add(0, t, (a @ WD[e].T) * wts[t, j].double()[:, None])
    O.backward(dout.double())
    for name, got, ref in [("out", out, O.detach()), ("dx", dxn, X.grad), ("dwg", dwg, WG.grad), ("dwu", dwu, WU.grad),
                           ("dwd", dwd, WD.grad)]:
        rel = ((got.double() - ref).norm() / ref.norm()).item()
        # at most eight bf16 roundings of 2^-9 in a chain
        assert rel < 2e-2, (name, rel)


def _all_calls(g, dtype=BF):
    x, w, dy = randn(g, 150, 256, dtype=dtype), randn(g, 192, 256, dtype=dtype, scale=0.06), randn(g, 150, 192, dtype=dtype)
    pre = randn(g, 150, 192, dtype=dtype)
    off, we = offsets_of([40, 0, 60, 50]), randn(g, 4, 192, 256, dtype=dtype, scale=0.06)
    mean, rstd = torch.zeros(150, device=DEV), torch.ones(150, device=DEV)
    one = x[:1].contiguous()

    def calls(stream=None):
        out = [moe.moe_layer_norm(x, stream=stream)]
        out += moe.moe_layer_norm_backward(x, x, None, mean, rstd, stream=stream)
        out += moe.moe_linear(x, w, None, dy, act="silu", want_pre=True, stream=stream)
        out += [moe.moe_linear(one, w, act="gelu", stream=stream)]
        out += moe.moe_linear_backward(dy, x, w, pre, act="gelu", want_dbias=True, stream=stream)
        out += [moe.moe_grouped_matmul(x, off, we, stream=stream), moe.moe_grouped_matmul_dgrad(dy, off, we, stream=stream),
                moe.moe_grouped_matmul_wgrad(dy, x, off, dtype=F32, stream=stream)]
        return out
    return calls, (x, w, dy, pre, we)


def test_repeatable_and_on_another_stream():
    calls, _ = _all_calls(gen(4))
    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        got = calls(stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    """Two graphs of the same calls, replayed in turn between eager calls, on inputs that change in place."""
    calls, inputs = _all_calls(gen(6))
    calls()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = calls()
        graphs.append((gr, out))
    for k in range(3):
        g = gen(100 + k)
        for t in inputs:
            t.copy_(randn(g, *t.shape, scale=0.5))
        want = [t.clone() for t in calls()]
        for gr, out in graphs:
            gr.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b), f"replay {k}"


def test_offsets_past_32_bits():
    """Rows behind 4 GiB of a strided matrix, and experts behind 4 GiB of weights."""
    g = gen(9)
    ld = 1 << 20
    big = torch.zeros(2200, ld, dtype=BF, device=DEV)
    x, w = big[:, :64], randn(g, 128, 64, scale=0.1)
    x.copy_(randn(g, 2200, 64))
    y = moe.moe_linear(x, w)
    assert torch.equal(y, moe.moe_linear(x.contiguous(), w))
    dy = randn(g, 2200, 128)
    a = moe.moe_linear_backward(dy, x, w)
    b = moe.moe_linear_backward(dy, x.contiguous(), w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    n = moe.moe_layer_norm(x)
    assert torch.equal(n, moe.moe_layer_norm(x.contiguous()))
    del big
    E, n_out, n_in = 200, 4096, 5120                # 8 GiB of weights
    we = torch.zeros(E, n_out, n_in, dtype=BF, device=DEV)
    we[E - 1] = randn(g, n_out, n_in, scale=0.02)
    xs, off = randn(g, 20, n_in), offsets_of([0] * (E - 1) + [20])
    # (one group alone may take another kernel than 200: another order of the same sums, so against 64 bits)
    X, W = xs.double(), we[E - 1].double()
    ref, acc = X @ W.T, 1.01 * n_in * ACC * X.abs() @ W.abs().T + tiny(BF)
    check(moe.moe_grouped_matmul(xs, off, we), ref, u(BF) * ref.abs() + acc, "y")
    d = randn(g, 20, n_out)
    assert torch.equal(moe.moe_grouped_matmul_dgrad(d, off, we), moe.moe_grouped_matmul_dgrad(d, offsets_of([20]), we[E - 1:]))
    dw = moe.moe_grouped_matmul_wgrad(d, xs, off)
    assert torch.equal(dw[E - 1:], moe.moe_grouped_matmul_wgrad(d, xs, offsets_of([20]))) and not dw[:E - 1].any()
