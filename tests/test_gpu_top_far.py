"""Log of the mass outside a list where exponents are far from 0 (temperatures of 1e-6 and below): finite wherever a column
outside the list is, in rows kept whole, streamed rows and rows cut into slices.

z / tau reaches 1e8 and more, so log-probs and rests are as large and are compared relative to themselves; tau is
given as the fp32 number that the call takes."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.choose_cases import close, dev_rows, tol_log
from tests.helpers import host
from tests.rules_cases import DTYPES, to_bits

pytestmark = pytest.mark.gpu


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tau", [1e-6, 1e-9])
@pytest.mark.parametrize("T,V,K", [(5, 5, 1), (5, 1000, 1), (5, 1000, 7), (5, 4000, 100), (5, 20011, 1), (5, 20011, 100),
                                   (5, 70001, 1), (5, 70001, 20), (5, 70001, 200), (1, 151936, 1)])
def test_rest_is_finite_where_columns_are_left(dtype, tau, T, V, K):
    tau = float(np.float32(tau))
    K = min(K, V - 1)
    rng = np.random.default_rng(V + K)
    z = rng.integers(100, 200, (T, V)) / 8.0
    for t in range(T):  # K values clear of all others, so that just K reach any floor
        z[t, rng.choice(V, K, replace=False)] = 30.0 + np.arange(K) / 8.0
    if T > 1:
        z[1] = 20.0  # all the same
        z[2, ::2] = -np.inf
    if T > 4:
        z[3, : V // 2] -= 40.0
        z[4] -= 60.0
    bits = to_bits(z, dtype)
    z = O.widen(bits, dtype)
    got = [host(g) for g in _lp().lp_top_logits(dev_rows(bits, dtype), K, None, tau)]
    want = O.top_logits(z, K, None, tau)
    assert np.array_equal(got[0], want[0])
    assert np.isfinite(want[2]).all()
    for g, w in zip(got[1:], want[1:]):
        close(g, w, tol_log(w, 2))
