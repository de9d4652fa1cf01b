"""Refusals of the layer norm, linear and grouped-product entry points, on the
CPU: bad sizes, types, strides, pointers and workspaces come back as errors
before anything is enqueued, and the binding refuses host tensors and shapes."""
import ctypes
import os

import pytest
import torch

import expert_ffn_dispatch_amd as moe
from expert_ffn_dispatch_amd import _lib

FAKE = 1 << 20          # an aligned address that is never dereferenced
INV, UNS, WSP = _lib.MOE_ERR_INVALID, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from expert_ffn_dispatch_amd import build
        build.build()
    return _lib.load()


def _err(lib):
    return lib.moe_last_error().decode()


def norm(**o):
    d = dict(rows=4, cols=64, dtype=0, param_dtype=0, flags=0, eps=1e-5, ld_x=0, ld_y=0, ld_dy=0, ld_dx=0)
    d.update(o)
    return _lib.MoeNormDims(*d.values())


def lin(**o):
    d = dict(rows=4, in_features=64, out_features=64, dtype=0, act=0, bias_dtype=0, dw_dtype=0, ld_x=0, ld_w=0,
             ld_residual=0, ld_y=0, ld_pre=0, ld_dy=0, ld_dx=0)
    d.update(o)
    return _lib.MoeLinearDims(*d.values())


def grp(**o):
    d = dict(rows=4, n_experts=2, in_features=64, out_features=64, dtype=0, dw_dtype=0, ld_x=0, ld_y=0)
    d.update(o)
    return _lib.MoeGroupedDims(*d.values())


@pytest.mark.parametrize("over,word", [
    (dict(rows=-1), "rows"), (dict(rows=(1 << 24) + 1), "rows"), (dict(cols=0), "cols"), (dict(cols=16385), "cols"),
    (dict(dtype=3), "dtype"), (dict(dtype=-1), "dtype"), (dict(param_dtype=1), "param_dtype"), (dict(flags=2), "flags"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(ld_x=63), "ld_x"), (dict(ld_y=-1), "ld_y"),
    (dict(ld_dy=(1 << 20) + 1), "ld_dy")])
def test_norm_dims(lib, over, word):
    d, n = norm(**over), ctypes.c_size_t(0)
    assert lib.moe_layer_norm(ctypes.byref(d), FAKE, None, None, FAKE, None, None, None) == INV and word in _err(lib)
    assert lib.moe_layer_norm_backward_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == INV
    assert lib.moe_layer_norm_backward(ctypes.byref(d), FAKE, FAKE, None, FAKE, FAKE, FAKE, None, None, None, 0, None) == INV


def test_norm_pointers(lib):
    d, r = norm(), ctypes.byref
    f, b = lib.moe_layer_norm, lib.moe_layer_norm_backward
    assert f(None, FAKE, None, None, FAKE, None, None, None) == INV and "dims" in _err(lib)
    assert f(r(d), None, None, None, FAKE, None, None, None) == INV and "x is NULL" in _err(lib)
    assert f(r(d), FAKE + 1, None, None, FAKE, None, None, None) == INV and "aligned" in _err(lib)
    assert f(r(d), FAKE, None, None, None, None, None, None) == INV and "y is NULL" in _err(lib)
    assert f(r(d), FAKE, None, None, FAKE, FAKE + 2, None, None) == INV and "mean" in _err(lib)
    assert f(r(norm(ld_x=80)), FAKE, None, None, FAKE, None, None, None) == INV and "stride" in _err(lib)
    assert b(r(d), FAKE, FAKE, None, None, FAKE, FAKE, None, None, None, 0, None) == INV and "mean" in _err(lib)
    assert b(r(d), FAKE, FAKE, None, FAKE, None, FAKE, None, None, None, 0, None) == INV and "rstd" in _err(lib)
    assert b(r(d), FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, None, None, 0, None) == WSP
    assert b(r(d), FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, None, FAKE + 16, 1 << 30, None) == WSP
    assert b(r(d), FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, None, FAKE, 16, None) == WSP
    # nothing to do: accepted without a launch
    assert f(r(norm(rows=0)), None, None, None, None, None, None, None) == 0
    assert b(r(d), FAKE, FAKE, None, FAKE, FAKE, None, None, None, None, 0, None) == 0


@pytest.mark.parametrize("over,code,word", [
    (dict(rows=-1), INV, "rows"), (dict(in_features=0), INV, "in_features"), (dict(out_features=65537), INV, "out_features"),
    (dict(dtype=2), INV, "dtype"), (dict(act=5), INV, "act"), (dict(bias_dtype=1), INV, "bias_dtype"),
    (dict(dw_dtype=1), INV, "dw_dtype"), (dict(ld_w=8), INV, "ld_w"), (dict(ld_pre=(1 << 20) + 1), INV, "ld_pre"),
    (dict(rows=1 << 24, out_features=65536, ld_residual=0), UNS, "tiles")])
def test_linear_dims(lib, over, code, word):
    d, n, r = lin(**over), ctypes.c_size_t(0), ctypes.byref
    assert lib.moe_linear_workspace_bytes(r(d), r(n)) == code and word in _err(lib)
    assert lib.moe_linear_backward_workspace_bytes(r(d), r(n)) == code
    assert lib.moe_linear(r(d), FAKE, 2 * FAKE, None, None, 3 * FAKE, None, FAKE, 1 << 40, None) == code
    assert lib.moe_linear_backward(r(d), FAKE, FAKE, FAKE, None, 2 * FAKE, None, None, FAKE, 1 << 40, None) == code


def test_linear_pointers(lib):
    d, r = lin(), ctypes.byref
    f, b = lib.moe_linear, lib.moe_linear_backward
    X, W, Y, Z = FAKE, 2 * FAKE, 3 * FAKE, 4 * FAKE
    assert f(r(d), None, W, None, None, Y, None, None, 0, None) == INV and "x is NULL" in _err(lib)
    assert f(r(d), X, W, None, None, X, None, None, 0, None) == INV and "output is an input" in _err(lib)
    assert f(r(d), X, W, None, None, Y, Y, None, 0, None) == INV
    assert f(r(d), X, W, None, Z, Y, Z, None, 0, None) == INV
    assert f(r(lin(ld_y=80)), X, W, None, Y, Y, None, None, 0, None) == INV and "stride" in _err(lib)
    assert f(r(lin(rows=100, in_features=4096)), X, W, None, None, Y, None, None, 0, None) == WSP
    assert f(r(lin(rows=0)), None, None, None, None, None, None, None, 0, None) == 0
    big = 1 << 40
    assert b(r(d), X, X, W, Z, Y, None, None, FAKE, big, None) == INV and "pre must be NULL" in _err(lib)
    assert b(r(lin(act=2)), X, X, W, None, Y, None, None, FAKE, big, None) == INV and "pre is NULL" in _err(lib)
    assert b(r(d), X, None, W, None, None, Y, None, FAKE, big, None) == INV and "x is NULL" in _err(lib)
    assert b(r(d), X, X, None, None, Y, None, None, FAKE, big, None) == INV and "w is NULL" in _err(lib)
    assert b(r(d), X, X, W, None, X, None, None, FAKE, big, None) == INV
    assert b(r(d), X, X, W, None, Y, None, None, None, 0, None) == WSP
    assert b(r(d), X, X, W, None, None, None, None, None, 0, None) == 0


@pytest.mark.parametrize("over,code,word", [
    (dict(rows=-1), INV, "rows"), (dict(n_experts=0), INV, "n_experts"), (dict(n_experts=257), UNS, "n_experts"),
    (dict(dtype=2), INV, "dtype"), (dict(dw_dtype=1), INV, "dw_dtype"), (dict(ld_x=1), INV, "ld_x"),
    (dict(ld_y=63), INV, "ld_y"), (dict(n_experts=256, in_features=65536, out_features=65536), UNS, "tiles")])
def test_grouped_dims(lib, over, code, word):
    d, n, r = grp(**over), ctypes.c_size_t(0), ctypes.byref
    X, W, Y = FAKE, 2 * FAKE, 3 * FAKE
    assert lib.moe_grouped_matmul(r(d), X, FAKE, W, Y, None) == code and word in _err(lib)
    assert lib.moe_grouped_matmul_dgrad(r(d), X, FAKE, W, Y, None) == code
    assert lib.moe_grouped_matmul_wgrad_workspace_bytes(r(d), r(n)) == code
    assert lib.moe_grouped_matmul_wgrad(r(d), X, X, FAKE, Y, FAKE, 1 << 40, None) == code


def test_grouped_pointers(lib):
    d, r = grp(), ctypes.byref
    X, W, Y = FAKE, 2 * FAKE, 3 * FAKE
    assert lib.moe_grouped_matmul(r(d), X, None, W, Y, None) == INV and "expert_offsets" in _err(lib)
    assert lib.moe_grouped_matmul(r(d), X, FAKE + 2, W, Y, None) == INV and "aligned" in _err(lib)
    assert lib.moe_grouped_matmul(r(d), X, FAKE, W, X, None) == INV
    assert lib.moe_grouped_matmul_dgrad(r(d), X, FAKE, None, Y, None) == INV
    assert lib.moe_grouped_matmul_wgrad(r(d), X, X, FAKE, X, FAKE, 1 << 40, None) == INV
    assert lib.moe_grouped_matmul_wgrad(r(grp(rows=4096)), X, X, FAKE, Y, None, 0, None) == WSP
    assert lib.moe_grouped_matmul(r(grp(rows=0)), None, None, None, None, None) == 0


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: moe.moe_layer_norm(x), lambda: moe.moe_linear(x, x), lambda: moe.moe_grouped_matmul(x, None, x),
                 lambda: moe.moe_layer_norm(None), lambda: moe.moe_linear_backward(x, x, x),
                 lambda: moe.moe_grouped_matmul_wgrad(x, x, None)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
