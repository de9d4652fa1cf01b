"""The sizes for which the GPU tests mean widened 4-bit weights are widened, on
the CPU: the workspace holds them."""
import pytest

import test_gpu_fp4_widened as wide
from test_more_operators_cpu import gat, grp, lib, lin, size  # noqa: F401


@pytest.mark.parametrize("rows,n_in,n_out,pad", wide.DENSE + [(*wide.EVERY, 0)])
def test_linear(lib, rows, n_in, n_out, pad):  # noqa: F811
    need = size(lib.moe_linear_fp4_workspace_bytes, lin(rows=rows, in_features=n_in, out_features=n_out, ld_x=n_in + pad))
    # rows at an odd pitch are copied behind the weights
    assert need >= 2 * n_in * n_out + (2 * rows * n_in if pad % 8 else 0)


@pytest.mark.parametrize("rows,n_in,width,pad", wide.GATED)
def test_gated(lib, rows, n_in, width, pad):  # noqa: F811
    need = size(lib.moe_gated_linear_fp4_workspace_bytes, gat(rows=rows, in_features=n_in, width=width, ld_x=n_in + pad))
    assert need >= 4 * n_in * width + (2 * rows * n_in if pad % 8 else 0)


@pytest.mark.parametrize("counts,n_in,n_out,pad", wide.GROUPED)
def test_grouped(lib, counts, n_in, n_out, pad):  # noqa: F811
    d = grp(rows=sum(counts), n_experts=len(counts), in_features=n_in, out_features=n_out, ld_x=n_in + pad)
    assert size(lib.moe_grouped_matmul_fp4_workspace_bytes, d) >= 2 * len(counts) * n_in * n_out


@pytest.mark.parametrize("counts,n_in,width,pad", wide.GROUPED_GATED)
def test_grouped_gated(lib, counts, n_in, width, pad):  # noqa: F811
    d = gat(rows=sum(counts), n_experts=len(counts), in_features=n_in, width=width, ld_x=n_in + pad)
    assert size(lib.moe_grouped_gated_fp4_workspace_bytes, d) >= 4 * len(counts) * n_in * width
