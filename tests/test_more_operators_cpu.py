"""Refusals of the gated projections, the AdamW step and the 4-bit products, on
the CPU: bad sizes, types, strides, pointers and workspaces come back as errors
before anything is enqueued, and the binding refuses host tensors.  Sizes of
workspaces: what is cut, copied or widened in the sizes that the GPU tests use."""
import ctypes
import os

import pytest
import torch

import expert_ffn_dispatch_amd as moe
import test_gpu_gated as gated
from expert_ffn_dispatch_amd import _lib
from test_abi_sanitized import _run, san_env  # noqa: F401
from test_operators_cpu import FAKE, INV, UNS, WSP, _err, grp, lib, lin  # noqa: F401

R = ctypes.byref
A, B, C, D, E, F, G, H = (FAKE * (i + 1) for i in range(8))      # addresses that are never dereferenced


def gat(**o):
    d = dict(rows=4, n_experts=1, in_features=64, width=64, dtype=0, act=4, dw_dtype=0, ld_x=0, ld_dx=0, ld_w=0, ld_h=0, ld_pre=0)
    d.update(o)
    return _lib.MoeGatedDims(*d.values())


def size(query, d):
    n = ctypes.c_size_t(0)
    assert query(R(d), R(n)) == 0
    return n.value


GATED_BAD = [
    (dict(rows=-1), INV, "rows"), (dict(rows=(1 << 24) + 1), INV, "rows"), (dict(in_features=0), INV, "in_features"),
    (dict(in_features=65537), INV, "in_features"), (dict(width=0), INV, "width"), (dict(width=65537), INV, "width"),
    (dict(dtype=2), INV, "dtype"), (dict(dtype=-1), INV, "dtype"), (dict(act=5), INV, "act"), (dict(act=-1), INV, "act"),
    (dict(dw_dtype=1), INV, "dw_dtype"), (dict(ld_x=63), INV, "ld_x"), (dict(ld_dx=-1), INV, "ld_dx"),
    (dict(ld_w=(1 << 20) + 1), INV, "ld_w"), (dict(ld_h=63), INV, "ld_h"), (dict(ld_pre=1), INV, "ld_pre"),
    (dict(n_experts=0), INV, "n_experts"), (dict(rows=1 << 24, width=65536), UNS, "tiles")]


@pytest.mark.parametrize("over,code,word", GATED_BAD)
def test_gated_dims(lib, over, code, word):  # noqa: F811
    d, n = gat(**over), ctypes.c_size_t(0)
    ws = (None, 0, None)
    for call in (lambda: lib.moe_gated_linear(R(d), A, B, C, D, None, None, *ws),
                 lambda: lib.moe_gated_linear_workspace_bytes(R(d), R(n)),
                 lambda: lib.moe_gated_linear_backward(R(d), A, B, C, D, E, F, G, None, None, *ws),
                 lambda: lib.moe_gated_linear_backward_workspace_bytes(R(d), R(n)),
                 lambda: lib.moe_gated_linear_fp4_workspace_bytes(R(d), R(n)),
                 lambda: lib.moe_grouped_gated(R(d), A, E, B, C, D, None, None, None),
                 lambda: lib.moe_grouped_gated_backward(R(d), A, B, H, C, D, E, F, G, None, None, *ws),
                 lambda: lib.moe_grouped_gated_backward_workspace_bytes(R(d), R(n)),
                 lambda: lib.moe_grouped_gated_fp4_workspace_bytes(R(d), R(n))):
        assert call() == code and word in _err(lib)


def test_gated_experts_and_strides(lib):  # noqa: F811
    n = ctypes.c_size_t(0)
    two = gat(n_experts=2)
    assert lib.moe_gated_linear_workspace_bytes(R(two), R(n)) == INV and "n_experts" in _err(lib)
    assert lib.moe_gated_linear(R(two), A, B, C, D, None, None, None, 0, None) == INV
    many = gat(n_experts=257)
    assert lib.moe_grouped_gated(R(many), A, E, B, C, D, None, None, None) == UNS and "n_experts" in _err(lib)
    wide = gat(n_experts=2, ld_w=72)
    assert lib.moe_grouped_gated(R(wide), A, E, B, C, D, None, None, None) == INV and "packed" in _err(lib)
    assert lib.moe_gated_linear_workspace_bytes(None, R(n)) == INV and "dims" in _err(lib)
    assert lib.moe_gated_linear_workspace_bytes(R(gat()), None) == INV and "bytes" in _err(lib)
    assert lib.moe_grouped_gated_backward_workspace_bytes(R(gat()), None) == INV and "bytes" in _err(lib)


def test_gated_pointers(lib):  # noqa: F811
    d = gat()
    f = lambda *a: lib.moe_gated_linear(R(d), *a, None, 0, None)  # noqa: E731
    assert lib.moe_gated_linear(None, A, B, C, D, None, None, None, 0, None) == INV and "dims" in _err(lib)
    assert f(None, B, C, D, None, None) == INV and "x is NULL" in _err(lib)
    assert f(A + 1, B, C, D, None, None) == INV and "aligned" in _err(lib)
    assert f(A, None, C, D, None, None) == INV and "w_gate is NULL" in _err(lib)
    assert f(A, B, None, D, None, None) == INV and "w_up is NULL" in _err(lib)
    assert f(A, B, C, None, None, None) == INV and "h is NULL" in _err(lib)
    assert f(A, B, C, D, E, None) == INV and "both" in _err(lib)
    assert f(A, B, C, D, None, E) == INV and "both" in _err(lib)
    assert f(A, B, C, A, None, None) == INV and "input" in _err(lib)
    assert f(A, B, C, D, B, E) == INV and "input" in _err(lib)
    assert f(A, B, C, D, D, E) == INV and "one" in _err(lib)
    assert f(A, B, C, D, E, E) == INV and "one" in _err(lib)
    assert lib.moe_grouped_gated(R(d), A, None, B, C, D, None, None, None) == INV and "expert_offsets is NULL" in _err(lib)
    assert lib.moe_grouped_gated(R(d), A, E + 2, B, C, D, None, None, None) == INV and "aligned" in _err(lib)
    big = gat(rows=300, in_features=4096)
    assert lib.moe_gated_linear(R(big), A, B, C, D, None, None, None, 0, None) == WSP
    assert f(*[None] * 6) == INV
    empty = gat(rows=0)
    assert lib.moe_gated_linear(R(empty), *[None] * 6, None, 0, None) == 0
    assert lib.moe_grouped_gated(R(empty), *[None] * 7, None) == 0


def test_gated_backward_pointers(lib):  # noqa: F811
    d = gat()
    need = size(lib.moe_gated_linear_backward_workspace_bytes, d)
    assert need >= 2 * 4 * 128
    W = 64 * FAKE
    f = lambda *a, ws=W, n=need: lib.moe_gated_linear_backward(R(d), *a, ws, n, None)  # noqa: E731
    good = [A, B, C, D, E, F, G, H, 9 * FAKE]                    # dh x w_gate w_up gate up dx dw_gate dw_up
    for i, word in enumerate(("dh", "x", "w_gate", "w_up", "gate", "up")):
        a = list(good)
        a[i] = None
        assert f(*a) == INV and f"{word} is NULL" in _err(lib)
        a[i] = good[i] + 1
        assert f(*a) == INV and "aligned" in _err(lib)
    assert f(*good[:8], None) == INV and "both" in _err(lib)
    assert f(*good[:7], None, good[8]) == INV and "both" in _err(lib)
    assert f(*good[:7], H, H) == INV and "one" in _err(lib)
    assert f(*good[:6], H, H, good[8]) == INV and "one" in _err(lib)
    for i in range(6):
        assert f(*good[:6], good[i], H, good[8]) == INV and "input" in _err(lib)
        assert f(*good[:7], good[i], good[8]) == INV and "input" in _err(lib)
    assert f(*good, ws=None) == WSP and f(*good, ws=W + 128) == WSP and f(*good, n=need - 1) == WSP
    g = lambda *a: lib.moe_grouped_gated_backward(R(d), *a, W, 1 << 40, None)  # noqa: E731
    assert g(A, B, None, C, D, E, F, G, None, None) == INV and "expert_offsets" in _err(lib)
    # nothing wanted: accepted without a launch
    assert f(*[None] * 9) == 0


@pytest.mark.parametrize("rows,n_in,width,side,cut", gated.CUT_TAILS)
def test_gated_forward_is_cut(lib, rows, n_in, width, side, cut):  # noqa: F811
    """Sizes that the GPU tests take for whole rounds of tiles and a cut tail (or none whole): partial tiles are what the
    workspace holds, a tile being `side` rows of half as many columns' gates and ups."""
    n = size(lib.moe_gated_linear_workspace_bytes, gat(rows=rows, in_features=n_in, width=width))
    tiles = -(-rows // side) * -(-2 * width // side)
    assert tiles % (256 if side == 256 else 512) == cut
    items, rest = divmod(n, side * side * 4)
    assert rest == 0 and items >= 2 * cut and items % cut == 0


# ----------------------------------------------------------- 4-bit products

def fp4(codes=A, exps=B + 1):
    return _lib.MoeFp4Matrix(codes, exps)


def test_fp4_widths_and_pointers(lib):  # noqa: F811
    n, m = ctypes.c_size_t(0), fp4()
    calls = {
        "linear": (lin, lambda d, x, w, y, *ws: lib.moe_linear_fp4(R(d), x, w, None, None, y, *ws), lib.moe_linear_fp4_workspace_bytes),
        "grouped": (grp, lambda d, x, w, y, *ws: lib.moe_grouped_matmul_fp4(R(d), x, H, w, y, *ws),
                    lib.moe_grouped_matmul_fp4_workspace_bytes),
        "gated": (gat, lambda d, x, w, y, *ws: lib.moe_gated_linear_fp4(R(d), x, R(m), w, y, *ws), lib.moe_gated_linear_fp4_workspace_bytes),
        "grouped gated": (gat, lambda d, x, w, y, *ws: lib.moe_grouped_gated_fp4(R(d), x, H, w, R(m), y, *ws),
                          lib.moe_grouped_gated_fp4_workspace_bytes)}
    for name, (dims, call, query) in calls.items():
        ws = (None, 0, None)
        for bad in (33, 48, 16, 1):
            d = dims(in_features=bad)
            assert call(d, C, R(m), D, *ws) == UNS and "32" in _err(lib), name
            assert query(R(d), R(n)) == UNS
        d = dims()
        assert query(R(d), None) == INV and "bytes" in _err(lib)
        assert query(None, R(n)) == INV and "dims" in _err(lib)
        assert call(d, None, R(m), D, *ws) == INV and "x is NULL" in _err(lib), name
        assert call(d, C + 1, R(m), D, *ws) == INV and "aligned" in _err(lib), name
        assert call(d, C, None, D, *ws) == INV and "NULL" in _err(lib), name
        assert call(d, C, R(fp4(codes=None)), D, *ws) == INV and "NULL" in _err(lib), name
        assert call(d, C, R(fp4(exps=None)), D, *ws) == INV and "NULL" in _err(lib), name
        assert call(d, C, R(fp4(codes=A + 8)), D, *ws) == INV and "16-byte" in _err(lib), name
        assert call(d, C, R(m), None, *ws) == INV and "NULL" in _err(lib), name
        assert call(d, C, R(m), C, *ws) == INV, name
        few, many = dims(rows=64, in_features=4096), dims(rows=1 << 17, in_features=4096)
        assert size(query, few) == 0, "the codes are read as they are"
        mats = 2 if "gated" in name else 1
        assert size(query, many) >= mats * 2 * 64 * 4096, "the weights are widened"
        assert call(many, C, R(m), D, *ws) == WSP, name
        assert call(dims(rows=0), None, None, None, *ws) == 0, name
    assert lib.moe_linear_fp4(R(lin(ld_w=96)), C, R(m), None, None, D, None, 0, None) == INV and "packed" in _err(lib)
    assert lib.moe_linear_fp4(R(lin(ld_residual=96)), C, R(m), None, D, D, None, 0, None) == INV and "stride" in _err(lib)
    assert lib.moe_linear_fp4(R(lin(act=7)), C, R(m), None, None, D, None, 0, None) == INV and "act" in _err(lib)


def test_quantise_fp4(lib):  # noqa: F811
    f = lambda w=A, dt=0, rows=4, cols=64, c=B, e=C: lib.moe_quantize_fp4(w, dt, rows, cols, c, e, None)  # noqa: E731
    for kw, word in ((dict(dt=2), "dtype"), (dict(dt=-1), "dtype"), (dict(rows=0), "rows"), (dict(rows=(1 << 26) + 1), "rows"),
                     (dict(cols=0), "cols"), (dict(cols=48), "cols"), (dict(cols=65568), "cols"), (dict(w=None), "w is NULL"),
                     (dict(w=A + 8), "16-byte"), (dict(c=None), "codes"), (dict(c=B + 4), "16-byte"), (dict(e=None), "exps")):
        assert f(**kw) == INV and word in _err(lib), kw


# -------------------------------------------------------------------- AdamW

def hyper(**o):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, flags=0, lr_device=None, step_device=None,
             grad_scale=None)
    d.update(o)
    return _lib.MoeAdamWArgs(*d.values())


def tensor(**o):
    d = dict(param=A, grad=B, exp_avg=C, exp_avg_sq=D, exp_avg_exp=None, exp_avg_sq_exp=None, copy=None, numel=8, param_dtype=2,
             grad_dtype=0, copy_dtype=0)
    d.update(o)
    return _lib.MoeAdamWTensor(*d.values())


def test_adamw_refusals(lib):  # noqa: F811
    nan, inf = float("nan"), float("inf")
    one = tensor()
    for kw, word in ((dict(lr=nan), "lr"), (dict(lr=inf), "lr"), (dict(weight_decay=nan), "weight_decay"), (dict(beta1=1.0), "beta1"),
                     (dict(beta1=-0.1), "beta1"), (dict(beta2=1.0), "beta2"), (dict(beta2=nan), "beta2"), (dict(eps=-1e-8), "eps"),
                     (dict(eps=inf), "eps"), (dict(step=0), "step"), (dict(step=-3), "step"), (dict(flags=2), "flags"),
                     (dict(lr_device=A + 2), "lr_device"), (dict(step_device=A + 1), "step_device"),
                     (dict(grad_scale=A + 3), "grad_scale")):
        assert lib.moe_adamw(R(hyper(**kw)), R(one), 1, None) == INV and word in _err(lib), kw
    ok = hyper()
    for kw, word in ((dict(numel=-1), "numel"), (dict(numel=(1 << 36) + 1), "numel"), (dict(param_dtype=3), "param_dtype"),
                     (dict(grad_dtype=-1), "grad_dtype"), (dict(copy=E, copy_dtype=2), "copy_dtype"), (dict(param=None), "param"),
                     (dict(param=A + 2), "param"), (dict(grad=B + 1), "grad"), (dict(exp_avg=None), "exp_avg"),
                     (dict(exp_avg_sq=None), "exp_avg"), (dict(exp_avg=C + 2), "exp_avg"), (dict(copy=E + 1), "copy"),
                     (dict(exp_avg=D), "one"), (dict(copy=A), "one"), (dict(grad=A, grad_dtype=2), "one")):
        both = (_lib.MoeAdamWTensor * 2)(tensor(numel=0), tensor(**kw))
        assert lib.moe_adamw(R(ok), both, 2, None) == INV and word in _err(lib), kw
        if word != "one":
            assert "1" in _err(lib) or word in ("param", "grad", "exp_avg", "copy"), "which tensor"
    assert lib.moe_adamw(R(hyper(flags=1)), R(one), 1, None) == INV and "exponents" in _err(lib)
    assert lib.moe_adamw(None, R(one), 1, None) == INV and "args" in _err(lib)
    assert lib.moe_adamw(R(ok), None, 1, None) == INV and "tensors" in _err(lib)
    assert lib.moe_adamw(R(ok), R(one), -1, None) == INV and "count" in _err(lib)
    # nothing to do: accepted without a launch
    assert lib.moe_adamw(R(ok), None, 0, None) == 0
    none = (_lib.MoeAdamWTensor * 2)(tensor(numel=0, param=None), tensor(grad=None))
    assert lib.moe_adamw(R(ok), none, 2, None) == 0
    assert lib.moe_adamw(R(hyper(step=0, step_device=A)), none, 2, None) == 0


# -------------------------------------------------------------- the binding

def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, 64, dtype=torch.bfloat16)
    off, w3 = torch.zeros(2, dtype=torch.int32), torch.zeros(1, 64, 64, dtype=torch.bfloat16)
    q = moe.Fp4Weights(torch.zeros(64, 32, dtype=torch.uint8), torch.zeros(64, 2, dtype=torch.uint8))
    q3 = moe.Fp4Weights(*(t[None] for t in q))
    for call in (lambda: moe.moe_gated_linear(x, w, w), lambda: moe.moe_grouped_gated(x, off, w3, w3),
                 lambda: moe.moe_gated_linear_backward(x, x, w, w, x, x), lambda: moe.moe_grouped_gated_backward(x, x, off, w3, w3, x, x),
                 lambda: moe.moe_linear_fp4(x, q), lambda: moe.moe_grouped_matmul_fp4(x, off, q3), lambda: moe.moe_gated_linear_fp4(x, q, q),
                 lambda: moe.moe_grouped_gated_fp4(x, off, q3, q3), lambda: moe.moe_quantize_fp4(w),
                 lambda: moe.AdamWTensors([x], [x], [x]), lambda: moe.moe_grouped_gated(x, None, w3, w3),
                 lambda: moe.moe_grouped_matmul_fp4(x, None, q3)):
        with pytest.raises(ValueError):
            call()


def test_values_of_4_bit_weights_and_8_bit_states():
    """The binding's own reading of the formats, against the definitions."""
    codes = torch.arange(256, dtype=torch.uint8).view(16, 16)
    exps = torch.arange(100, 116, dtype=torch.uint8)[:, None]
    v = moe.Fp4Weights(codes, exps).values()
    mag = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for r in range(16):
        for j in range(32):
            c = (int(codes[r, j // 2]) >> (4 * (j % 2))) & 15
            assert v[r, j].item() == (-1) ** (c >> 3) * mag[c & 7] * 2.0 ** (int(exps[r, 0]) - 127)
    m = moe.Fp8Moment.zeros(torch.empty(300))
    assert m.codes.shape == (300,) and m.exps.shape == (3,) and not m.values().any()
    m.codes.view(torch.uint8)[:] = 0x38                          # 1.0
    m.exps[:] = torch.tensor([127, 1, 255], dtype=torch.uint8)
    w = m.values()
    assert (w[:128] == 1).all() and (w[128:256] == 2.0 ** -126).all() and torch.isnan(w[256:]).all()


@pytest.mark.skipif("MOE_FFN_LIB" in os.environ, reason="inside the run below")
def test_under_sanitizers(san_env):  # noqa: F811
    """The argument checks above against the build whose host code runs under the sanitizers."""
    r = _run(san_env, ["-m", "pytest", "tests/test_more_operators_cpu.py", "-q", "-p", "no:cacheprovider"])
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error:" not in r.stderr, tail
