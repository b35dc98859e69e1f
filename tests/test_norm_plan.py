"""The gradients of a norm leave one row of partial parameter gradients per workgroup: no more of them
than there are sets of rows for a workgroup (the size of the workspace, on the CPU)."""
import pytest

import selective_state_space_20_amd as sss

# rows that one workgroup of 256 lanes takes at once, in the smaller of the shapes for bf16 and fp32
ROWS = [(4, 32), (64, 16), (128, 8), (256, 4), (512, 4), (1024, 1)]


@pytest.mark.parametrize("n, at_once", ROWS)
@pytest.mark.parametrize("rows", [1, 31, 97, 200, 500, 1000])
@pytest.mark.parametrize("groups", [1, 3])
def test_no_workgroup_without_rows(n, at_once, rows, groups):
    sets = -(-rows // at_once)
    assert sss.rms_norm_gated_bwd_workspace_size(rows, n * groups, n) <= sets * n * groups * 4
    if groups == 1:
        assert sss.rms_norm_residual_bwd_workspace_size(rows, n) <= sets * 3 * n * 4
