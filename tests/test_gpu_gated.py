"""Gated projections, dense and by expert, with their gradients, against the
formulas in 64 bits.  Tolerances count roundings as in test_gpu_operators.py;
the operands of the gradients' products are rounded to the data's type first,
which adds u sum|a b| for each."""
import math

import pytest
import torch

import expert_ffn_dispatch_amd as moe
import test_gpu_operators as T
from test_gpu_operators import (ACC, ACTS, BF, DEV, F32, FUN, HF, act_grad_ref, act_ref, check, gen, offsets_of, randn,
                                strided, tiny, u)

pytestmark = pytest.mark.gpu


def check_forward(x, wg, wu, act, h, gate, up, what=""):
    dt = x.dtype
    X, G, U = x.double(), wg.double(), wu.double()
    zg, zu = X @ G.T, X @ U.T
    eg = 1.01 * (x.shape[1] + 2) * ACC * X.abs() @ G.abs().T
    eu = 1.01 * (x.shape[1] + 2) * ACC * X.abs() @ U.abs().T
    if gate is not None:
        check(gate, zg, u(dt) * zg.abs() + eg + tiny(dt), what + " gate")
        check(up, zu, u(dt) * zu.abs() + eu + tiny(dt), what + " up")
    a = act_ref(zg, act)
    ea = 1.2 * eg + FUN * a.abs() + ACC * zg.abs()          # slopes of the activations are at most 1.13
    ref = a * zu
    err = ea * (zu.abs() + eu) + a.abs() * eu + 2 * ACC * ref.abs()
    check(h, ref, u(dt) * ref.abs() + 1.01 * err + tiny(dt), what + " h")


def grads_ref(dh, gate, up, act):
    """dgate, dup in 64 bits, and how far the kernel's operands may be from them."""
    dt = dh.dtype
    D, Z, U = dh.double(), gate.double(), up.double()
    s, a = act_grad_ref(Z, act), act_ref(Z, act)
    dg, du = D * U * s, D * a
    fun = 0 if act in ("none", "relu") else FUN
    eg = (u(dt) + 3 * ACC) * dg.abs() + fun * (D * U).abs() + tiny(dt)
    eu = (u(dt) + 3 * ACC) * du.abs() + fun * (D.abs() * (a.abs() + Z.abs())) + tiny(dt)
    return dg, du, eg, eu


def check_backward(dh, x, wg, wu, gate, up, act, dx, dwg, dwu, what=""):
    dt, rows, width = dh.dtype, dh.shape[0], dh.shape[1]
    dg, du, eg, eu = grads_ref(dh, gate, up, act)
    X, G, U = x.double(), wg.double(), wu.double()
    if dx is not None:
        ref = dg @ G + du @ U
        n = 2 * (width + 64)                                 # one contraction over both, in whole stages
        err = (eg + n * ACC * dg.abs()) @ G.abs() + (eu + n * ACC * du.abs()) @ U.abs()
        check(dx, ref, u(dt) * ref.abs() + 1.01 * err + tiny(dt), what + " dx")
    for got, d, e, name in ((dwg, dg, eg, "dw_gate"), (dwu, du, eu, "dw_up")):
        ref = d.T @ X
        err = (e + (rows + 2) * ACC * d.abs()).T @ X.abs()
        check(got, ref, u(got.dtype) * ref.abs() + 1.01 * err + tiny(got.dtype), what + " " + name)


# rows, in, width: one token, few rows, odd widths, ragged tiles, contraction slices, several rounds
SHAPES = [(1, 64, 64), (1, 2048, 520), (3, 1, 1), (2, 7, 5), (17, 72, 40), (37, 512, 256), (64, 1000, 136), (33, 256, 6200),
          (130, 264, 392), (129, 65, 131), (300, 4096, 64), (257, 768, 512), (1, 4097, 33), (700, 1001, 1003),
          (333, 1003, 96), (100, 2048, 768)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,n_in,width", SHAPES)
def test_forward(rows, n_in, width, act):
    g = gen(rows + n_in + width)
    dt = HF if (rows + width) % 2 else BF
    x = randn(g, rows, n_in, dtype=dt)
    wg, wu = (randn(g, width, n_in, dtype=dt, scale=n_in ** -0.5) for _ in range(2))
    h, gate, up = moe.moe_gated_linear(x, wg, wu, act=act, want_pre=True)
    check_forward(x, wg, wu, act, h, gate, up)
    assert torch.equal(moe.moe_gated_linear(x, wg, wu, act=act), h)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,n_in,width", SHAPES)
def test_backward(rows, n_in, width, act):
    g = gen(rows + 3 * n_in + width)
    dt = BF if (rows + width) % 2 else HF
    x, dh = randn(g, rows, n_in, dtype=dt), randn(g, rows, width, dtype=dt)
    wg, wu = (randn(g, width, n_in, dtype=dt, scale=n_in ** -0.5) for _ in range(2))
    gate, up = randn(g, rows, width, dtype=dt, scale=2.0), randn(g, rows, width, dtype=dt)
    dx, dwg, dwu = moe.moe_gated_linear_backward(dh, x, wg, wu, gate, up, act=act, dw_dtype=F32 if act == "relu" else None)
    check_backward(dh, x, wg, wu, gate, up, act, dx, dwg, dwu)
    only = moe.moe_gated_linear_backward(dh, x, wg, wu, gate, up, act=act, want_dw=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    only = moe.moe_gated_linear_backward(dh, x, wg, wu, gate, up, act=act, want_dx=False, dw_dtype=dwg.dtype)
    assert only[0] is None and torch.equal(only[1], dwg) and torch.equal(only[2], dwu)


# rows, in, width, side of the tiles, tiles that are cut (all of them, or those behind whole rounds over the card)
CUT_TAILS = [(300, 4096, 64, 128, 3), (4400, 4400, 2200, 256, 68), (4200, 2048, 2052, 256, 33), (2100, 4160, 2100, 128, 49)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("rows,n_in,width", [c[:3] for c in CUT_TAILS] + [(4001, 520, 2171)])
def test_whole_rounds_and_a_cut_tail(rows, n_in, width, act):
    """The products are saved and joined partly in the tiles, partly where the slices are added."""
    g = gen(rows)
    x, dh = randn(g, rows, n_in), randn(g, rows, width)
    wg, wu = (randn(g, width, n_in, scale=n_in ** -0.5) for _ in range(2))
    h, gate, up = moe.moe_gated_linear(x, wg, wu, act=act, want_pre=True)
    check_forward(x, wg, wu, act, h, gate, up)
    check_backward(dh, x, wg, wu, gate, up, act, *moe.moe_gated_linear_backward(dh, x, wg, wu, gate, up, act=act))


def test_gradient_against_differences():
    g = gen(11)
    x, dh = randn(g, 6, 24), randn(g, 6, 16)
    wg, wu = randn(g, 16, 24, scale=0.2), randn(g, 16, 24, scale=0.2)
    for act in ACTS:
        gate, up = (x.double() @ w.double().T for w in (wg, wu))
        gate, up = gate.to(BF), up.to(BF)
        dx, dwg, dwu = moe.moe_gated_linear_backward(dh, x, wg, wu, gate, up, act=act, dw_dtype=F32)
        h, D, Z, U = 1e-5, dh.double(), gate.double(), up.double()
        dg = D * U * (act_ref(Z + h, act) - act_ref(Z - h, act)) / (2 * h)
        du = D * act_ref(Z, act)
        eg, eu = u(BF) * dg.abs() + 1e-5 * (D * U).abs(), u(BF) * du.abs() + 1e-5 * D.abs()
        ref = dg @ wg.double() + du @ wu.double()
        check(dx, ref, u(BF) * ref.abs() + 1.01 * (eg @ wg.double().abs() + eu @ wu.double().abs()) + 1e-6, "dx " + act)
        for got, d, e in ((dwg, dg, eg), (dwu, du, eu)):
            check(got, d.T @ x.double(), 1.01 * e.T @ x.double().abs() + 1e-5, "dw " + act)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", ACTS[1:])
def test_activation_at_large_values(act, dtype):
    """Far out the activation is the gate or 0 and its slope 1 or 0, exactly."""
    top = float(torch.finfo(dtype).max)
    z = torch.tensor([129.0, 300.0, 1e4, 6e4, min(1e20, top), top, top / 3, 200.0], device=DEV).to(dtype)
    z = torch.stack([z, -z])
    eye, one = torch.eye(8, dtype=dtype, device=DEV), torch.ones(2, 8, dtype=dtype, device=DEV)
    h, gate, up = moe.moe_gated_linear(torch.cat([z, one], 1), torch.cat([eye, 0 * eye], 1), torch.cat([0 * eye, eye], 1),
                                       act=act, want_pre=True)
    assert torch.equal(gate, z) and torch.equal(up, one) and torch.equal(h, z.clamp(min=0))
    dx = moe.moe_gated_linear_backward(one, one, eye, 0 * eye, z, one, act=act)[0]
    assert torch.equal(dx, (z > 0).to(dtype))
    # dup = dh act(gate)
    dx = moe.moe_gated_linear_backward(one, one, 0 * eye, eye, z, one, act=act)[0]
    assert torch.equal(dx, z.clamp(min=0))


# gate, up, dh
PAST = [(-math.inf, 1, 1), (-math.inf, 2, 0), (-math.inf, -math.inf, 1), (-300, math.inf, 1), (-300, -math.inf, 2), (math.inf, 3, 1),
        (math.inf, 2, 0), (-2, math.inf, 0), (math.inf, math.inf, 1), (0.5, math.inf, 1), (0.5, math.nan, 0), (-300, 1, math.nan),
        (-300, math.nan, 1), (math.nan, 1, 1), (1, -2, 0), (-300, 3, 1)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", ACTS)
def test_saved_products_past_the_type(act, dtype):
    """A saved product that is infinite stands for a finite sum past the type's range (fp16: 65504): its gradient is the limit,
    0 where the other factor is 0, infinite elsewhere, and no number only where an operand is none.  One row of ones as x:
    the weights' gradients are dgate and dup."""
    z, up, d = (torch.tensor([c[i] for c in PAST], device=DEV).to(dtype)[None] for i in range(3))
    x, w = torch.ones(1, 8, dtype=dtype, device=DEV), torch.zeros(len(PAST), 8, dtype=dtype, device=DEV)
    _, dg, du = moe.moe_gated_linear_backward(d, x, w, w, z, up, act=act, want_dx=False)
    for i, (zi, ui, di) in enumerate(PAST):
        far = zi if act == "none" else max(zi, 0.0) if zi == zi else zi          # act(gate), past |gate| = 128
        slope = 1.0 if act == "none" else float(zi > 0) if zi == zi or act == "relu" else zi
        if abs(zi) < 128:
            far, slope = act_ref(z[0, i].double(), act).item(), act_grad_ref(z[0, i].double(), act).item()
        for got, saved, factor in ((dg, ui, di * slope), (du, far, di)):
            want = 0.0 if factor == 0 and abs(saved) == math.inf else saved * factor
            have = got[i, 0].item()
            assert (have != have) == (want != want) and (want != want or have == want or (
                math.isfinite(want) and abs(have - want) <= 2 * u(dtype) * abs(want) + 2 * FUN)), (PAST[i], have, want)


@pytest.mark.parametrize("act", ACTS[1:])
def test_gates_below_the_types_range(act):
    """A gate sum of -80000 in fp16: h is 0, the saved gate -inf, and the step has no gradient through it."""
    x = torch.tensor([[40000.0, 1.0], [1.0, 1.0]], device=DEV).to(HF)
    wg, wu = torch.tensor([[-2.0, 0.0], [0.0, 1.0]], device=DEV).to(HF), torch.tensor([[0.0, 1.0], [0.0, 2.0]], device=DEV).to(HF)
    h, gate, up = moe.moe_gated_linear(x, wg, wu, act=act, want_pre=True)
    assert h[0, 0] == 0 and gate[0, 0] == -math.inf
    dh = torch.tensor([[1.0, 0.0], [0.0, 1.0]], device=DEV).to(HF)
    dx, dwg, dwu = moe.moe_gated_linear_backward(dh, x, wg, wu, gate, up, act=act)
    assert not dx[0].any() and not dwg[0].any() and not dwu[0].any()
    assert torch.isfinite(dx).all() and torch.isfinite(dwg).all() and torch.isfinite(dwu).all()


@pytest.mark.parametrize("n_in,width,pad,shift", [(128, 192, 8, 0), (128, 192, 3, 0), (136, 72, 16, 8), (96, 64, 8, 1),
                                                  (77, 51, 2, 3)])
@pytest.mark.parametrize("rows", [5, 70, 150])
def test_strides(rows, n_in, width, pad, shift):
    g = gen(n_in)
    x, dh = randn(g, rows, n_in), randn(g, rows, width)
    wg, wu = randn(g, width, n_in, scale=0.1), randn(g, width, n_in, scale=0.1)
    S = lambda t: strided(t, pad, shift)  # noqa: E731
    outs = [S(torch.zeros_like(dh)) for _ in range(3)]
    moe.moe_gated_linear(S(x), S(wg), S(wu), h=outs[0], gate=outs[1], up=outs[2])
    check_forward(x, wg, wu, "silu", *outs)
    _, gate, up = (t.contiguous() for t in outs)
    dx = S(torch.zeros_like(x))
    got = moe.moe_gated_linear_backward(S(dh), S(x), S(wg), S(wu), S(gate), S(up), dx=dx)
    check_backward(dh, x, wg, wu, gate, up, "silu", *got)
    for t in outs + [dx]:
        pads = t._base.reshape(-1)[shift:].view(rows, t.shape[1] + pad)[:, t.shape[1]:]
        assert torch.isnan(pads).all(), "the space between rows was written"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,n_in,width", T.GROUPS, ids=[f"{len(c)}x{sum(c)}-{i}-{o}" for c, i, o in T.GROUPS])
def test_grouped(counts, n_in, width, dtype):
    g = gen(sum(counts) + n_in)
    front, back = 3, 5                              # rows outside every group
    E, rows = len(counts), sum(counts) + front + back
    off = offsets_of(counts, front)
    x, dh = randn(g, rows, n_in, dtype=dtype), randn(g, rows, width, dtype=dtype)
    wg, wu = (randn(g, E, width, n_in, dtype=dtype, scale=n_in ** -0.5) for _ in range(2))
    for t in (x, dh):
        t[:front] = float("nan")
        t[rows - back:] = float("nan")
    for e, c in enumerate(counts):
        if c == 0:
            wg[e] = wu[e] = float("nan")            # never read
    h, gate, up = (torch.full((rows, width), 7.0, dtype=dtype, device=DEV) for _ in range(3))
    dx = torch.full((rows, n_in), 7.0, dtype=dtype, device=DEV)
    moe.moe_grouped_gated(x, off, wg, wu, h=h, gate=gate, up=up)
    outs = [moe.moe_grouped_gated_backward(dh, x, off, wg, wu, gate, up, dx=dx),
            moe.moe_grouped_gated_backward(dh, x, off, wg, wu, gate, up, want_dx=False, dw_dtype=F32)]
    for t in (h, gate, up, dx):
        assert (t[:front] == 7).all() and (t[rows - back:] == 7).all(), "rows outside the groups were written"
    b = front
    for e, c in enumerate(counts):
        s = slice(b, b + c)
        if c:
            check_forward(x[s], wg[e], wu[e], "silu", h[s], gate[s], up[s], f"{e}")
        for dxs, dwg, dwu in outs:
            if c == 0:
                assert not dwg[e].any() and not dwu[e].any()
            else:
                check_backward(dh[s], x[s], wg[e], wu[e], gate[s], up[s], "silu", dxs[s] if dxs is not None else None,
                               dwg[e], dwu[e], f"{e}")
        b += c


def test_offsets_are_clamped_and_empty():
    g = gen(8)
    x, dh, wg, wu = randn(g, 40, 64), randn(g, 40, 72), randn(g, 3, 72, 64), randn(g, 3, 72, 64)
    gate, up = randn(g, 40, 72), randn(g, 40, 72)
    bad = torch.tensor([-5, 10, 7, 1000], dtype=torch.int32, device=DEV)
    h = moe.moe_grouped_gated(x, bad, wg, wu)
    # expert 0 has rows 0..9, expert 1 none, expert 2 rows 7..39
    assert torch.equal(h[:7], moe.moe_grouped_gated(x[:10], offsets_of([10, 0, 0]), wg, wu)[:7])
    assert torch.equal(h[10:], moe.moe_grouped_gated(x[7:], offsets_of([0, 0, 33]), wg, wu)[3:])
    dx, dwg, dwu = moe.moe_grouped_gated_backward(dh, x, bad, wg, wu, gate, up, dw_dtype=F32)
    assert not dwg[1].any() and not dwu[1].any()
    for lo, hi, e in ((0, 10, 0), (7, 40, 2)):
        s = slice(lo, hi)
        check_backward(dh[s], x[s], wg[e], wu[e], gate[s], up[s], "silu", None, dwg[e], dwu[e], f"{e}")
    e64, e72 = torch.empty(0, 64, dtype=BF, device=DEV), torch.empty(0, 72, dtype=BF, device=DEV)
    zero = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert moe.moe_grouped_gated(e64, zero, wg, wu).shape == (0, 72)
    dx, dwg, dwu = moe.moe_grouped_gated_backward(e72, e64, zero, wg, wu, e72, e72)
    assert dx.shape == (0, 64) and not dwg.any() and not dwu.any()
    assert moe.moe_gated_linear(e64, wg[0], wu[0]).shape == (0, 72)
    dx, dwg, dwu = moe.moe_gated_linear_backward(e72, e64, wg[0], wu[0], e72, e72)
    assert dx.shape == (0, 64) and not dwg.any() and not dwu.any()


def test_not_a_number_stays_in_its_row():
    g = gen(9)
    for rows in (20, 150):
        x, wg, wu = randn(g, rows, 64), randn(g, 80, 64), randn(g, 80, 64)
        want = moe.moe_gated_linear(x, wg, wu)
        x[3, 1] = float("nan")
        h = moe.moe_gated_linear(x, wg, wu)
        ok = torch.arange(rows, device=DEV) != 3
        assert torch.equal(h[ok], want[ok]) and torch.isnan(h[3]).all()


def _calls(g):
    x, dh = randn(g, 150, 256), randn(g, 150, 192)
    wg, wu = randn(g, 192, 256, scale=0.06), randn(g, 192, 256, scale=0.06)
    eg, eu, off = randn(g, 4, 192, 256, scale=0.06), randn(g, 4, 192, 256, scale=0.06), offsets_of([40, 0, 60, 50])
    gate, up, one = randn(g, 150, 192), randn(g, 150, 192), x[:1].contiguous()

    def calls(stream=None):
        out = [*moe.moe_gated_linear(x, wg, wu, want_pre=True, stream=stream), moe.moe_gated_linear(one, wg, wu, stream=stream)]
        out += moe.moe_gated_linear_backward(dh, x, wg, wu, gate, up, act="gelu", stream=stream)
        out += moe.moe_grouped_gated(x, off, eg, eu, want_pre=True, stream=stream)
        out += moe.moe_grouped_gated_backward(dh, x, off, eg, eu, gate, up, dw_dtype=F32, stream=stream)
        return out
    return calls, (x, dh, wg, wu, eg, eu, gate, up)


def test_repeatable_and_on_another_stream():
    calls, _ = _calls(gen(4))
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
    calls, inputs = _calls(gen(6))
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


def test_as_the_two_products_apart():
    """The saved products are the ones that moe_grouped_matmul computes, and h is moe_grouped_ffn's intermediate: the
    down projection of it is that call's output, up to the order of fp32 sums (a rounding step of h, then of y)."""
    g = gen(12)
    E, M, H = 4, 256, 192
    off, x = offsets_of([100, 0, 30, 70]), randn(g, 200, M)
    wg, wu, wd = randn(g, E, H, M, scale=M ** -0.5), randn(g, E, H, M, scale=M ** -0.5), randn(g, E, M, H, scale=H ** -0.5)
    h, gate, up = moe.moe_grouped_gated(x, off, wg, wu, want_pre=True)
    for got, w in ((gate, wg), (up, wu)):
        ref = moe.moe_grouped_matmul(x, off, w).double()
        check(got, ref, 2 * u(BF) * ref.abs() + 1e-5, "product")
    y = moe.moe_grouped_matmul(h, off, wd)
    ffn = moe.moe_grouped_ffn(moe.dims(200, M, E, 1, H), x, off, wg, wu, wd)
    assert ((y.float() - ffn.float()).norm() / ffn.float().norm()).item() < 2 * 2.0 ** -8


def test_offsets_past_32_bits():
    """Experts behind 4 GiB of weights, rows behind 4 GiB of a strided matrix."""
    g = gen(9)
    E, width, n_in = 200, 4096, 5120
    wg, wu = (torch.zeros(E, width, n_in, dtype=BF, device=DEV) for _ in range(2))
    wg[E - 1], wu[E - 1] = randn(g, width, n_in, scale=0.02), randn(g, width, n_in, scale=0.02)
    xs, off = randn(g, 20, n_in), offsets_of([0] * (E - 1) + [20])
    h, gate, up = moe.moe_grouped_gated(xs, off, wg, wu, want_pre=True)
    check_forward(xs, wg[E - 1], wu[E - 1], "silu", h, gate, up)
    dh = randn(g, 20, width)
    got = moe.moe_grouped_gated_backward(dh, xs, off, wg, wu, gate, up)
    check_backward(dh, xs, wg[E - 1], wu[E - 1], gate, up, "silu", got[0], got[1][E - 1], got[2][E - 1])
    assert not got[1][:E - 1].any() and not got[2][:E - 1].any()
    del wg, wu, got
    ld = 1 << 20
    big = torch.zeros(2200, ld, dtype=BF, device=DEV)
    x, wa, wb = big[:, :64], randn(g, 128, 64, scale=0.1), randn(g, 128, 64, scale=0.1)
    x.copy_(randn(g, 2200, 64))
    out = moe.moe_gated_linear(x, wa, wb, want_pre=True)
    for a, b in zip(out, moe.moe_gated_linear(x.contiguous(), wa, wb, want_pre=True)):
        assert torch.equal(a, b)
    dh = randn(g, 2200, 128)
    for a, b in zip(moe.moe_gated_linear_backward(dh, x, wa, wb, out[1], out[2]),
                    moe.moe_gated_linear_backward(dh, x.contiguous(), wa, wb, out[1], out[2])):
        assert torch.equal(a, b)
