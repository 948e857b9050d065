"""How a state and its result are walked, on the host."""
import pytest
import torch

import entropy_chunked_row_amd as lp


@pytest.mark.parametrize("shape,dim", [((2, 0, 6, 3), 2), ((0, 2, 6, 3), 2), ((2, 6, 0), 1), ((6, 4, 0, 5), 0), ((3, 0, 6), 2)])
def test_states_without_an_element_are_walked(shape, dim):
    outer, _, _, mid, _, width = lp._state_layout(torch.zeros(shape), dim, "state")
    assert outer * mid * width == 0


def test_layouts():
    t = torch.zeros(2, 6, 3, 9)
    assert lp._state_layout(t, 1, "state") == (2, 6 * 27 * 4, 27 * 4, 1, 0, 27 * 4)
    assert lp._state_layout(t[..., :8], 1, "state") == (2, 6 * 27 * 4, 27 * 4, 3, 9 * 4, 8 * 4)
    assert lp._state_layout(t[:, :, :2, :8], 1, "state") == (2, 6 * 27 * 4, 27 * 4, 2, 9 * 4, 8 * 4)
