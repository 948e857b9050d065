"""States and results of different layouts: dense into a prefix of each row of a larger cache, the other way round, and
states without an element."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.helpers import host, to_dev

pytestmark = pytest.mark.gpu
PARENTS = [[[2, 0, 0], [1, 1, 2]], [[0, 1, 2, 2, 0], [1, -1, 1, 3, 1]]]


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


@pytest.mark.parametrize("dtype", ["uint8", "int16", "float32", "int64"])
@pytest.mark.parametrize("shape,dim", [((6, 3, 9), 0), ((2, 6, 3, 16), 1), ((6, 2, 3, 8), 0), ((6, 3, 1), 0), ((6, 1, 9), 0),
                                       ((3, 6, 5, 1000), 1), ((1, 6, 4, 64), 1)])
@pytest.mark.parametrize("par", PARENTS, ids=["as many", "more"])
def test_dense_and_prefix(dtype, shape, dim, par):
    import torch
    rng = np.random.default_rng(3)
    p = np.array(par, dtype=np.int32)
    a = rng.integers(-100 if dtype != "uint8" else 0, 100, shape).astype(dtype)
    want = O.beam_reorder(a, p, dim)
    state = to_dev(a)
    wide = list(want.shape)
    wide[-1] += 5
    for src in (state, torch.nn.functional.pad(state, (0, 3))[..., :shape[-1]]):
        assert np.array_equal(host(_lp().lp_beam_reorder(src, to_dev(p), dim=dim)), want)
        buf = torch.full(wide, 9, dtype=state.dtype, device="cuda")
        got = _lp().lp_beam_reorder(src, to_dev(p), dim=dim, out=buf[..., :shape[-1]])
        assert got.data_ptr() == buf.data_ptr() and np.array_equal(host(got), want) and bool((buf[..., shape[-1]:] == 9).all())
        dense = torch.full(want.shape, 9, dtype=state.dtype, device="cuda")
        assert np.array_equal(host(_lp().lp_beam_reorder(src, to_dev(p), dim=dim, out=dense)), want)


def test_layouts_that_share_no_walk_are_refused():
    import torch
    p = to_dev(np.array(PARENTS[0], dtype=np.int32))
    state = torch.zeros(6, 4, 3, 8, device="cuda")[:, :, :2]             # 4 parts of 16
    out = torch.zeros(6, 4, 2, 9, device="cuda")[..., :8]                # 8 parts of 8
    with pytest.raises(ValueError, match="walked"):
        _lp().lp_beam_reorder(state, p, out=out)


@pytest.mark.parametrize("shape,dim", [((2, 0, 6, 3), 2), ((0, 2, 6, 3), 2), ((2, 6, 0), 1), ((6, 4, 0, 5), 0), ((6, 0, 4, 5), 0),
                                       ((3, 0, 6), 2)])
def test_states_without_an_element(shape, dim):
    import torch
    p = to_dev(np.array(PARENTS[1], dtype=np.int32))
    want = list(shape)
    want[dim] = 10
    state = torch.zeros(shape, device="cuda")
    assert list(_lp().lp_beam_reorder(state, p, dim=dim).shape) == want
    out = torch.zeros(want, device="cuda")
    assert _lp().lp_beam_reorder(state, p, dim=dim, out=out) is out
