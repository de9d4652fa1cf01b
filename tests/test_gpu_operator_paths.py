"""Layer norm, linear layers and products grouped by expert on the paths that
calls of ordinary sizes take, against the formulas in 64 bits.  Tolerances
count roundings as in test_gpu_operators.py."""
import ctypes
import math

import pytest
import torch

import expert_ffn_dispatch_amd as moe
from expert_ffn_dispatch_amd import _lib
from test_gpu_operators import ACC, BF, DEV, F32, check, gen, randn, u

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
