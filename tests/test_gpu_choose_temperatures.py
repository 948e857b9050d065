"""Temperatures far from one: which continuations beams take, and the gradient of distillation."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.choose_cases import close, dev_rows, grad_tol, lists, peaked, tol_log
from tests.helpers import host, to_dev
from tests.rules_cases import DTYPES

pytestmark = pytest.mark.gpu
TAU = [float(np.float32(t)) for t in (1e-4, 0.02, 30.0, 1e6)]


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tau", TAU)
@pytest.mark.parametrize("V", [900, 12007, 70001])
def test_beams(dtype, tau, V):
    """Each continuation has the score that it is given, none comes twice, a beam's come in the order of its logits, and
    none better is left out: which beam is first is free only where two scores are closer than a log-sum is known."""
    rng = np.random.default_rng(3)
    B, W, N = 2, 3, 7
    bits, z = peaked(rng, B * W, V, dtype)
    s = np.zeros((B, W), dtype=np.float32)
    scores, parents, tokens = [host(t) for t in _lp().lp_beam_select(dev_rows(bits, dtype), to_dev(s), N, None, 0, tau)]
    best, pa, to = O.beam_select(z, s, N, None, 0, tau)
    close(scores, best, tol_log(best, 2))
    logp = O.log_softmax(O.tempered(z, tau))
    for b in range(B):
        at = logp[b * W + parents[b], tokens[b]]
        close(scores[b], at, tol_log(at, 2))
        assert len(set(zip(parents[b], tokens[b]))) == N
        for w in range(W):
            own = tokens[b][parents[b] == w]
            assert np.array_equal(own, O._top_order(z[b * W + w])[:own.size])
        more, _, _ = O.beam_select(z[b * W:(b + 1) * W], s[:1], N + 1, None, 0, tau)
        other = O.beam_select(z[b * W:(b + 1) * W], s[:1], N + 1, None, 0, tau)[1][0]
        gap = more[0, :-1] - more[0, 1:]
        if np.all((gap > 2 * np.max(tol_log(more, 2))) | (other[:-1] == other[1:])):
            assert np.array_equal(parents[b], pa[b]) and np.array_equal(tokens[b], to[b])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tau", TAU)
@pytest.mark.parametrize("V", [900, 12007, 70001])
def test_gradient(dtype, tau, V):
    """grad_tol counts the rounding of log-sums of z / tau, which the gradient's probabilities are taken from."""
    lp = _lp()
    rng = np.random.default_rng(5)
    bits, z = peaked(rng, 6, V, dtype)
    ids, lpk, rest = lists(rng, z, 11, 1.0)
    x, a = dev_rows(bits, dtype), [to_dev(t) for t in (ids, lpk, rest)]
    _, lse, lse_rest = lp.lp_distill_top(x, *a, None, tau)
    g = np.linspace(-1, 1, 6).astype(np.float32) * np.float32(min(tau, 1.0))
    d = lp.lp_distill_top_backward(x, *a, None, tau, lse, lse_rest, to_dev(g))
    ref = O.distill_top_backward(z, ids, lpk, rest, None, tau, g)
    close(host(d.float()), ref, grad_tol(z, ids, lpk, rest, tau, g, ref, dtype))
