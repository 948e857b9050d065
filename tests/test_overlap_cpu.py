"""C entry points refuse outputs and workspaces that share bytes with an
operand, before anything is launched (addresses are never dereferenced)."""
import pytest

A = 1 << 20  # an address, and room between operands
FAR = 1 << 30


@pytest.mark.parametrize("off,ld,ld_out", [(16, 16, 16), (15, 32, 32), (17, 32, 32), (31, 40, 40), (48, 32, 40),
                                           (32 * 3 + 15, 32, 32), (-15, 32, 32), (-17, 32, 32)])
def test_rules_outputs(lib_handle, off, ld, ld_out):
    """4 rows of 16 bf16 columns, the output `off` columns behind the logits."""
    L = lib_handle
    h = (A, 0, 4, 16, ld, None)
    assert L.lp_process_logits(*h, None, A + 2 * off, ld_out, None) == 1
    assert L.lp_processed_logprobs_entropy_backward(*h, FAR, None, 1.0, FAR, None, FAR, None, A + 2 * off, ld_out,
                                                    None) == 1
