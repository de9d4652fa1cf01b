"""Workspaces: the alignment that the header states is the one that every entry
point asks for, on the CPU (a workspace at half of it is refused before
anything is enqueued)."""
import ctypes
import os
import re

import pytest

import expert_ffn_dispatch_amd as moe
from expert_ffn_dispatch_amd import _lib
from test_operators_cpu import grp, lib, lin, norm  # noqa: F401

FAKE = 1 << 20          # an address that is never dereferenced
BIG = 1 << 40
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_ffn.h")


def stated():
    with open(HEADER) as f:
        return int(re.search(r"#define MOE_WORKSPACE_ALIGN (\d+)", f.read()).group(1))


def test_header_states_one_alignment():
    with open(HEADER) as f:
        text = re.sub(r"\s*\n \*\s*", " ", f.read())
    assert "All pointers must be 16-byte aligned, workspaces MOE_WORKSPACE_ALIGN bytes" in text
    assert "workspaces MOE_WORKSPACE_ALIGN bytes as above" in text
    assert not re.search(r"workspace\w* \d+ bytes", text)


@pytest.mark.parametrize("part", [2, 4, 16])
def test_entry_points_ask_for_it(lib, part):  # noqa: F811
    r = ctypes.byref
    ws = FAKE + stated() // part
    X, W, Y = FAKE, 2 * FAKE, 3 * FAKE
    d = moe.dims(64, 64, 4, 2, 64)
    n, l, g = norm(), lin(rows=100, in_features=4096), grp(rows=4096)
    calls = {
        "moe_route": lambda: lib.moe_route(r(d), X, W, None, Y, Y, ws, BIG, None),
        "moe_layer_norm_backward": lambda: lib.moe_layer_norm_backward(r(n), X, X, None, X, X, Y, Y, None, ws, BIG, None),
        "moe_linear": lambda: lib.moe_linear(r(l), X, W, None, None, Y, None, ws, BIG, None),
        "moe_linear_backward": lambda: lib.moe_linear_backward(r(l), X, X, W, None, Y, None, None, ws, BIG, None),
        "moe_grouped_matmul_wgrad": lambda: lib.moe_grouped_matmul_wgrad(r(g), X, X, FAKE, Y, ws, BIG, None),
    }
    for name, call in calls.items():
        assert call() == _lib.MOE_ERR_WORKSPACE, name
        assert f"{stated()}-byte aligned" in lib.moe_last_error().decode(), name
