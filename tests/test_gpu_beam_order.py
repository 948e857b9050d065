"""Within a beam its logits decide, also where the score so far is so large, or the temperature so high, that the sums are
equal: no token comes before one of a larger logit of its own beam."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.choose_cases import close, dev_rows, peaked, tol_log
from tests.helpers import host, to_dev
from tests.rules_cases import DTYPES, to_bits

pytestmark = pytest.mark.gpu


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,N", [(50, 8), (5003, 8), (5003, 100), (70001, 8)])
@pytest.mark.parametrize("far", [-1e20, float(np.finfo(np.float32).min)])
def test_scores_that_take_up_every_logit(dtype, V, N, far):
    """Beams of a score that stands for none (a finite one): they fill the places that the others leave."""
    rng = np.random.default_rng(V + N)
    B, W = 3, 3
    bits, z = peaked(rng, B * W, V, dtype)
    z = z.copy()
    z[0, 5:] = -np.inf            # a grammar leaves the only live beam five tokens
    z[3] = np.where(np.arange(V) % 2 == 0, z[3], -np.inf)
    z[6:9] = z[6]                 # equal rows, equal scores: the lowest beam, its largest logits
    bits = to_bits(z, dtype)
    z = O.widen(bits, dtype)
    s = np.full((B, W), far, dtype=np.float32)
    s[0, 0] = -1.0
    s[1, 1:] = -np.inf
    got = [host(g) for g in _lp().lp_beam_select(dev_rows(bits, dtype), to_dev(s), N)]
    with np.errstate(invalid="ignore"):
        want = O.beam_select(z, s, N, None, 0, 1.0)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[2], want[2])
    close(got[0], want[0], tol_log(want[0]))
    for b, w in ((0, 1), (1, 0), (2, 0)):
        own = got[2][b][got[1][b] == w]
        row = z[b * W + w]
        assert own.size and np.array_equal(own, O._top_order(row)[:own.size])


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_temperature_that_levels_every_logit(dtype):
    rng = np.random.default_rng(1)
    V, N, tau = 9001, 12, float(np.float32(1e30))
    bits, z = peaked(rng, 2, V, dtype)
    s = np.array([[0.0], [-3.0]], dtype=np.float32)
    got = [host(g) for g in _lp().lp_beam_select(dev_rows(bits, dtype), to_dev(s), N, None, 0, tau)]
    want = O.beam_select(z, s, N, None, 0, tau)
    for b in range(2):
        assert np.array_equal(got[2][b], O._top_order(z[b])[:N]) and not got[1][b].any()
    close(got[0], want[0], tol_log(want[0]))
