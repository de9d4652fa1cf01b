"""Layer norm, linear layers and products grouped by expert on the paths that
calls of ordinary sizes take, against the formulas in 64 bits.  Tolerances
count roundings as in test_gpu_operators.py."""
import ctypes
import math

import pytest
import torch

import expert_ffn_dispatch_amd as moe
from expert_ffn_dispatch_amd import _lib
import test_gpu_operators as T
from test_gpu_operators import ACC, BF, DEV, F32, check, gen, offsets_of, randn, u

pytestmark = pytest.mark.gpu


def call(fn, query, d, args, ws):
    """A C entry point with a workspace of the caller's."""
    n = ctypes.c_size_t(0)
    _lib.check(query(ctypes.byref(d), ctypes.byref(n)))
    assert n.value <= ws.numel()
    _lib.check(fn(ctypes.byref(d), *args, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream))


@pytest.mark.parametrize("offsets", [[1000, 2500, 2500, 5000, 6000], [0, 20000, 20000, 20000, 20000], [7] * 5, [6000, 100, 4000, 50, 9000]])
def test_weight_gradient_leaves_rows_outside_the_groups_unread(offsets):
    """Odd widths: the operands are copied with padded rows, the rows of the groups alone."""
    g = gen(sum(offsets))
    rows, E, n_in, n_out = 20000, 4, 1001, 1003
    x, dy = randn(g, rows, n_in), randn(g, rows, n_out)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    dw = torch.empty(E, n_out, n_in, device=DEV)
    d = _lib.MoeGroupedDims(rows, E, n_in, n_out, _lib.MOE_DTYPE_BF16, _lib.MOE_DTYPE_F32, 0, 0)
    lib = _lib.load()
    ws = torch.full((1 << 28,), 0x5A, dtype=torch.uint8, device=DEV)
    call(lib.moe_grouped_matmul_wgrad, lib.moe_grouped_matmul_wgrad_workspace_bytes, d,
         (dy.data_ptr(), x.data_ptr(), off.data_ptr(), dw.data_ptr()), ws)
    spans = []
    for e in range(E):
        lo = offsets[e]
        spans.append((lo, max(lo, offsets[e + 1])))
    first, end = min(lo for lo, _ in spans), max(hi for _, hi in spans)
    # rows of 1024 at the front of the workspace: dy's copy, then x's
    copies = ws[:2 * rows * 2048].view(torch.int16).view(2, rows, 1024)
    for t, w in ((copies[0], dy), (copies[1], x)):
        assert torch.equal(t[first:end, :w.shape[1]], w[first:end].view(torch.int16)), "the operands are not copied as this test takes it"
        assert (t[:first] == 0x5A5A).all() and (t[end:] == 0x5A5A).all(), "rows outside the groups were read"
    for e, (lo, hi) in enumerate(spans):
        D, X = dy[lo:hi].double(), x[lo:hi].double()
        ref = D.T @ X
        check(dw[e], ref, 2.0 ** -24 * ref.abs() + (hi - lo + 1) * ACC * D.abs().T @ X.abs() + 1e-30, f"dw {e}")


# ------------------------------------------------------------------- gelu

def normal(z):
    """Distribution and density in 64 bits, the distribution without 1 + erf."""
    return 0.5 * torch.special.erfc(-z * 0.5 ** 0.5), torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5


def gelu_rel(z):
    """Relative error of the distribution and density in fp32: the tail's eight powers 2^-20, the fast exponential of
    z^2 / 2 twice 2^-24 of its argument, and four roundings."""
    return 2.0 ** -20 + (z * z / 2 + 4) * 2.0 ** -23


@pytest.mark.parametrize("rows", [50, 400])
def test_gelu_keeps_its_bits_far_out(rows):
    """Values from -12.5 to 12.5, down to 1e-34, each within its rounding (the kernels for few rows and of tiles)."""
    z = torch.linspace(-12.5, 12.5, rows * 16, device=DEV).to(BF).view(rows, 16)
    y = moe.moe_linear(z, torch.eye(16, dtype=BF, device=DEV), act="gelu")
    Z = z.double()
    ref = Z * normal(Z)[0]
    check(y, ref, (u(BF) + gelu_rel(Z)) * ref.abs(), "gelu")


def test_gelu_slope_keeps_its_bits_far_out():
    """The bias gradient of one row is the slope itself, in fp32."""
    n = 4000
    z = torch.linspace(-12.5, 12.5, n, device=DEV).to(BF)[None]
    one = torch.ones_like(z)
    dx, dw, db = moe.moe_linear_backward(one, z[:, :8].contiguous(), one.view(n, 1).expand(n, 8).contiguous(), z, act="gelu",
                                         want_dx=False, want_dw=False, want_dbias=True, bias_dtype=F32)
    assert dx is None and dw is None
    Z = z[0].double()
    P, p = normal(Z)
    check(db, P + Z * p, gelu_rel(Z) * (P + Z.abs() * p), "slope")


# ------------------------------------------------------------------- norm

@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [3, 33, 100, 264])
def test_norm_gradient_of_far_rows(cols, dtype, rms):
    """A row of one value near the top of the range: n is 0 at every column, though -mean * rstd overflows; with the
    root-mean-square form, whose mean is 0, a NaN mean is ignored."""
    g = gen(cols)
    far = 1.5 * 2.0 ** 120
    x, dy, gamma = randn(g, 5, cols, dtype=dtype), randn(g, 5, cols, dtype=dtype), randn(g, cols, dtype=F32)
    x[2] = 0.0 if rms else far
    mean = torch.full((5,), float("nan"), device=DEV) if rms else x.float().mean(1)
    if not rms:
        mean[2] = far
    rstd = torch.full((5,), 300.0, device=DEV)
    dx, dgamma, dbeta = moe.moe_layer_norm_backward(dy, x, gamma, mean, rstd, rms=rms)
    D, r = dy.double(), 300.0
    n = (x.double() - (0 if rms else mean.double()[:, None])) * r
    gg = D * gamma.double()
    ref = r * (gg - (0 if rms else gg.mean(1, keepdim=True)) - n * (gg * n).mean(1, keepdim=True))
    mag = r * (gg.abs() + gg.abs().mean(1, keepdim=True) + n.abs() * (gg * n).abs().mean(1, keepdim=True))
    # sums of up to 264 terms and six roundings a term, each of n's own size (|x - mean| is exact to 2^-23 of |x| + |mean|)
    en = 4 * ACC * (x.double().abs() + (0 if rms else mean.double().abs()[:, None])) * r
    en[2] = 0
    far_n = r * en * (gg * n).abs().mean(1, keepdim=True) + r * n.abs() * (gg.abs() * en).mean(1, keepdim=True)
    check(dx, ref, u(dtype) * ref.abs() + (cols + 8) * ACC * mag + 2 * far_n, "dx")
    acc = (cols + 8) * ACC
    check(dgamma, (D * n).sum(0), acc * (D * n).abs().sum(0) + (D.abs() * en).sum(0) + 1e-30, "dgamma")
    check(dbeta, D.sum(0), acc * D.abs().sum(0) + 1e-30, "dbeta")


def test_norm_gradient_in_place_and_in_part():
    """dx in the place of dy or x, and calls that leave outputs out, give the same values bit for bit."""
    for rows, cols, dtype in ((300, 640, BF), (1000, 2048, F32), (37, 5121, BF), (5, 16384, torch.float16), (130, 8200, F32)):
        g = gen(cols)
        x, dy, gamma = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols, dtype=dtype), randn(g, cols, dtype=dtype)
        for rms in (False, True):
            _, mean, rstd = moe.moe_layer_norm(x, gamma, rms=rms, want_stats=True)
            f = lambda a, b, **o: moe.moe_layer_norm_backward(a, b, gamma, mean, rstd, rms=rms, **o)  # noqa: E731
            want = f(dy, x)
            for i in range(2):
                a, b = dy.clone(), x.clone()
                got = f(a, b, dx=(a, b)[i])
                assert got[0] is (a, b)[i] and all(torch.equal(p, q) for p, q in zip(got, want)), (cols, i)
                assert torch.equal((b, a)[i], (x, dy)[i])
            dx, dga, dbe = f(dy, x, want_params=False)
            assert torch.equal(dx, want[0]) and dga is None and dbe is None
            dx, dga, dbe = f(dy, x, want_dx=False)
            assert dx is None and torch.equal(dga, want[1]) and torch.equal(dbe, want[2])
            assert f(dy, x, want_dx=False, want_params=False) == (None, None, None)


# ---------------------------------------------------------- linear layers

# Forward products whose tile lists are whole rounds over the card and a part of one, which is cut along the contraction
# (rows, in, out; tiles of a side; tiles cut).  test_operator_plans_cpu.py holds the plans to this.
CUT_TAILS = [(4400, 4400, 4400, 256, 68), (4200, 2048, 4104, 256, 33), (2100, 4160, 4200, 128, 49)]


@pytest.mark.parametrize("act", T.ACTS)
@pytest.mark.parametrize("rows,n_in,n_out", [c[:3] for c in CUT_TAILS])
def test_linear_whole_rounds_and_a_cut_tail(rows, n_in, n_out, act):
    """Bias, activation, residual and z partly in the tiles, partly in the join."""
    T.test_linear_forward(rows, n_in, n_out, act)


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("rows,n_in,n_out", [(4400, 4400, 4400), (2100, 1032, 4200)])
def test_linear_gradients_of_several_rounds(rows, n_in, n_out, act):
    T.test_linear_backward(rows, n_in, n_out, act)


def test_linear_residual_in_place_with_a_cut_tail():
    rows, n_in, n_out = CUT_TAILS[0][:3]
    g = gen(rows)
    x, w, r = randn(g, rows, n_in), randn(g, n_out, n_in, scale=n_in ** -0.5), randn(g, rows, n_out)
    want = moe.moe_linear(x, w, None, r, act="silu")
    y = r.clone()
    assert torch.equal(moe.moe_linear(x, w, None, y, act="silu", y=y), want)


# 17 to 64 rows with 32 and 64 columns to a block, sixteen rows of many columns
@pytest.mark.parametrize("rows,n_in,n_out", [(16, 264, 12400), (17, 1032, 6200), (32, 256, 12400), (20, 8, 12289), (49, 1544, 6150),
                                             (64, 520, 6200), (50, 1032, 12290), (64, 136, 16384)])
@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
def test_linear_few_rows_of_many_columns(rows, n_in, n_out, act):
    T.test_linear_forward(rows, n_in, n_out, act)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_odd_widths_of_several_rounds(act):
    """A contraction too short for padded copies: unaligned tiles, more of them than blocks."""
    T.test_linear_forward(3000, 9, 5001, act)
    T.test_linear_backward(3000, 9, 5001, act)


@pytest.mark.parametrize("shift", [1, 4])
def test_linear_misaligned_and_cut(shift):
    """Pointers that do not suit 16-byte loads though the strides do: unaligned tiles, cut along the contraction."""
    g = gen(shift)
    rows, n_in, n_out = 130, 2048, 200
    x, w, r, dy = randn(g, rows, n_in), randn(g, n_out, n_in, scale=n_in ** -0.5), randn(g, rows, n_out), randn(g, rows, n_out)
    S = lambda t: T.strided(t, 8, shift)  # noqa: E731
    X, W, D = x.double(), w.double(), dy.double()
    y, pre = moe.moe_linear(S(x), S(w), None, S(r), act="silu", want_pre=True)
    z, ez = X @ W.T, 1.01 * (n_in + 2) * ACC * X.abs() @ W.abs().T
    check(pre, z, u(BF) * z.abs() + ez + T.tiny(BF), "pre")
    ref = T.act_ref(z, "silu") + r.double()
    check(y, ref, u(BF) * ref.abs() + 1.2 * ez + T.FUN * z.abs() + 2 * ACC * ref.abs() + T.tiny(BF), "y")
    dx, dw, db = moe.moe_linear_backward(S(dy), S(x), S(w), want_dbias=True, dw_dtype=F32, bias_dtype=F32)
    check(dx, D @ W, u(BF) * (D @ W).abs() + 1.01 * n_out * ACC * D.abs() @ W.abs() + T.tiny(BF), "dx")
    check(dw, D.T @ X, u(F32) * (D.T @ X).abs() + 1.01 * rows * ACC * D.abs().T @ X.abs(), "dw")
    check(db, D.sum(0), u(F32) * D.sum(0).abs() + (rows + 8) * ACC * D.abs().sum(0), "dbias")


@pytest.mark.parametrize("rows,n_in,n_out,act", [(130, 264, 392, "gelu"), (65, 1001, 1003, "silu"), (1000, 512, 2056, "none")])
def test_linear_gradients_in_part(rows, n_in, n_out, act):
    """Calls that leave outputs out, or name dx's place, give the same values bit for bit."""
    g = gen(rows)
    x, w, dy, pre = randn(g, rows, n_in), randn(g, n_out, n_in, scale=0.05), randn(g, rows, n_out), randn(g, rows, n_out)
    pre = None if act == "none" else pre
    want = moe.moe_linear_backward(dy, x, w, pre, act=act, want_dbias=True)
    for bits in range(8):
        ask = [bool(bits >> i & 1) for i in range(3)]
        got = moe.moe_linear_backward(dy, x, w, pre, act=act, want_dx=ask[0], want_dw=ask[1], want_dbias=ask[2])
        for q, a, b in zip(ask, got, want):
            assert (a is None) if not q else torch.equal(a, b)
    place = T.strided(torch.zeros_like(x), 24)
    got = moe.moe_linear_backward(dy, x, w, pre, act=act, want_dw=False, dx=place)[0]
    assert got is place and torch.equal(place, want[0])


# -------------------------------------------------------- products by expert

RAGGED = [0, 700, 33, 260, 1, 511, 300, 0, 900, 257, 129, 64, 290, 513, 31, 777]


@pytest.mark.parametrize("dtype", [BF, torch.float16])
def test_grouped_large_tiles(dtype):
    """256 x 256 tiles of unequal groups, more of them than blocks, forward and back: some waves' rows are in part or
    not at all live, and each form's blocks take a second tile."""
    n_in, n_out, mean = 2312, 2296, sum(RAGGED) // len(RAGGED)
    tiles = sum(-(-c // 256) for c in RAGGED) * -(-n_out // 256)
    assert mean > 256 and len(RAGGED) * 2 * (n_out // 256) >= 192 and tiles > 256
    T.test_grouped(RAGGED, n_in, n_out, dtype)


@pytest.mark.parametrize("n_in,n_out", [(520, 640), (515, 643), (600, 519)])
def test_grouped_more_tiles_than_blocks(n_in, n_out):
    """128 x 128 tiles, aligned and of odd widths, in several rounds over the card."""
    counts = [(7 * e * e) % 97 for e in range(200)]
    assert sum(-(-c // 128) for c in counts) * 5 > 512
    T.test_grouped(counts, n_in, n_out, BF)


# Weight gradients of several groups whose tiles are cut along the rows, and whose blocks take several tiles
GROUPED_CUT = ([20000, 0, 12700, 68], 512, 512)


@pytest.mark.parametrize("dtype", [BF, torch.float16])
def test_grouped_weight_gradient_cut(dtype):
    T.test_grouped(*GROUPED_CUT, dtype)


def test_grouped_weight_gradient_of_several_rounds():
    T.test_grouped([100, 0, 300, 65, 7], 2304, 2048, BF)


# ----------------------------------------------------------------- together

def test_large_calls_repeat_and_run_side_by_side():
    """The same inputs give the same bits: again, with the caches overwritten in between, and two at once."""
    g = gen(77)
    x, w, dy = randn(g, 4000, 2560), randn(g, 5120, 2560, scale=0.02), randn(g, 4000, 5120)
    counts = [(13 * e * e) % 301 + 200 for e in range(16)]
    off = offsets_of(counts)
    rows = sum(counts)
    xs, ds, we = randn(g, rows, 2560), randn(g, rows, 1536), randn(g, 16, 1536, 2560, scale=0.02)

    def calls():
        y, pre = moe.moe_linear(x, w, act="gelu", want_pre=True)
        out = [y, pre, *moe.moe_linear_backward(dy, x, w, pre, act="gelu", want_dbias=True)]
        out += [moe.moe_grouped_matmul(xs, off, we), moe.moe_grouped_matmul_dgrad(ds, off, we),
                moe.moe_grouped_matmul_wgrad(ds, xs, off, dtype=F32)]
        y, mean, rstd = moe.moe_layer_norm(x, want_stats=True)
        return out + [y, *moe.moe_layer_norm_backward(x, x, None, mean, rstd)]

    want = calls()
    cache = torch.empty(1 << 29, dtype=torch.uint8, device=DEV)
    for k in range(3):
        cache.fill_(k)
        assert all(torch.equal(a, b) for a, b in zip(calls(), want)), k
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    both = []
    for s in streams:
        with torch.cuda.stream(s):
            both.append(calls())
    torch.cuda.synchronize()
    for got in both:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
