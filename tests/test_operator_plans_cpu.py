"""The shapes that test_gpu_operator_paths.py runs still take the paths it names,
on the CPU: partial tiles of cut products are what their workspace holds."""
import ctypes

import pytest

import test_gpu_operator_paths as paths
from test_operators_cpu import grp, lib, lin  # noqa: F401


def cut_tiles(nbytes, side):
    """Slices times tiles of a workspace that holds only partial tiles, or None."""
    n, rest = divmod(nbytes, side * side * 4)
    return n if rest == 0 else None


@pytest.mark.parametrize("rows,n_in,n_out,side,cut", paths.CUT_TAILS)
def test_forward_cut_tails(lib, rows, n_in, n_out, side, cut):  # noqa: F811
    d, n = lin(rows=rows, in_features=n_in, out_features=n_out), ctypes.c_size_t(0)
    assert lib.moe_linear_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == 0
    tiles = -(-rows // side) * -(-n_out // side)
    slots = 256 if side == 256 else 512
    assert tiles > slots and tiles % slots == cut
    items = cut_tiles(n.value, side)
    assert items is not None and items >= 2 * cut and items % cut == 0


def test_grouped_weight_gradient_cut(lib):  # noqa: F811
    counts, n_in, n_out = paths.GROUPED_CUT
    d, n = grp(rows=sum(counts) + 8, n_experts=len(counts), in_features=n_in, out_features=n_out), ctypes.c_size_t(0)
    assert lib.moe_grouped_matmul_wgrad_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == 0
    items = cut_tiles(n.value, 128)
    tiles = len(counts) * (n_in // 128) * (n_out // 128)
    assert items is not None and items >= 2 * tiles and items % tiles == 0


def test_misaligned_pointers_are_cut(lib):  # noqa: F811
    d, n = lin(rows=130, in_features=2048, out_features=200, ld_x=2056, ld_w=2056), ctypes.c_size_t(0)
    assert lib.moe_linear_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == 0
    assert n.value >= 2 * 4 * 128 * 128 * 4
