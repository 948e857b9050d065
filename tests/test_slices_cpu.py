"""Which rows of logits are cut into slices, seen through the workspace that a call asks for."""
import pytest


@pytest.mark.parametrize("dtype,longest", [(0, 65536), (1, 65536), (2, 32768)])
@pytest.mark.parametrize("T,K", [(4, 5), (1, 20), (16, 200), (100, 64)])
def test_rows_past_128_kilobytes_are_cut(lib_handle, dtype, longest, T, K):
    assert lib_handle.lp_top_workspace_bytes(dtype, T, longest, K) == 256
    assert lib_handle.lp_top_workspace_bytes(dtype, T, longest + 1, K) > 256
    assert lib_handle.lp_top_workspace_bytes(dtype, 5000, 200000, K) == 256  # many rows are not
