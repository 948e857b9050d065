"""Scoring under logit rules at the far ends of the number range, against the
fp64 oracle.

Tolerances, derived before the first run.  An exponent t = (z - m) log2(e) / tau
that still weighs anything is at least -150; it is one fp32 operation (two where
|m log2(e) / tau| passes 2^24), so off by at most 150 * 2^-23 = 1.8e-5 where its
weight is 2^-150, and by t 2^t 2^-23 < 1e-7 in the sum.  What is left is the
target's own exponent, up to |t| = 64 of the normal logits here: 64 * 2^-24
ln 2, and the sums' roundings: 1e-5, the bar of the other logits calls.  The
log-sum-exp is as large as the logits: 2^-22 relative (the rounded log2(e) / tau,
the product, the sum, the factor ln 2: half a step of 2^-24 relative each)."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.helpers import host, to_dev, to_dev_bits
from tests.rules_cases import EPS, to_bits

pytestmark = pytest.mark.gpu
TOL = 1e-5
LOWEST = {"bf16": -3.3895313892515355e38, "fp32": -3.4028234663852886e38, "fp16": -65504.0}


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def _dev(x, dtype):
    b = to_bits(x, dtype)
    return (to_dev(b) if dtype == "fp32" else to_dev_bits(b, dtype)), O.widen(b, dtype)


def _wide(t):
    return host(t.float()).astype(np.float64)


def _check_scores(got, z, y, tau):
    want = O.logprobs_entropy(z, y, None, tau)
    for g, w in zip(got[:2], want[:2]):
        assert np.abs(host(g) - w).max() <= TOL
    lse = np.asarray(want[2])
    assert np.all(np.abs(host(got[2]) - lse) <= TOL + 2.0 ** -22 * np.abs(lse))


def _check_grad(d, z, slope, y, tau, g, gh, dtype):
    want = O.processed_backward(z, slope, y, None, tau, g, gh)
    logp = O.log_softmax(O.tempered(z, tau))
    p = np.exp(logp)
    size = (np.abs(g) + np.abs(gh))[:, None] * (1 + p * (np.abs(np.maximum(logp, -1e4)) + 12))
    tol = EPS[dtype] / 2 * np.abs(want) + 2 * TOL * size * np.abs(slope) / tau + 2.0 ** -25
    assert np.all(np.abs(d - want) <= tol)


@pytest.mark.parametrize("T,V", [(6, 20011), (800, 5003)], ids=["slices", "whole_rows"])
@pytest.mark.parametrize("tau", [0.7, 1.0, 1.5, 2.0])
@pytest.mark.parametrize("dtype,low", [("bf16", -1e10), ("bf16", -1e30), ("bf16", -1e38), ("bf16", LOWEST["bf16"]),
                                       ("fp32", -1e10), ("fp32", -1e30), ("fp32", -1e38), ("fp32", LOWEST["fp32"]),
                                       ("fp16", LOWEST["fp16"])])
def test_finite_masks_weigh_nothing(T, V, tau, dtype, low):
    """Finite mask values in whole lanes, whole slices and all of a row but a
    few columns, ahead of the real logits and behind them."""
    rng = np.random.default_rng(V)
    x = rng.normal(0, 3, (T, V))
    y = rng.integers(0, V, T).astype(np.int64)
    keep = rng.random((T, V)) < 0.5
    keep[0::6] = np.arange(V) >= V - 60
    keep[1::6] = np.arange(V) < 45
    keep[2::6] = np.arange(V) >= V // 2
    keep[3::6] = np.arange(V) // 64 % 2 == 1
    keep[np.arange(T), y] = True
    x, z = _dev(np.where(keep, x, low), dtype)
    lp = _lp()
    got = lp.lp_processed_logprobs_entropy(x, None, to_dev(y), None, tau)
    _check_scores(got, z, y, tau)
    g, gh = rng.normal(0, 1, T).astype(np.float32), rng.normal(0, 0.5, T).astype(np.float32)
    d = _wide(lp.lp_processed_logprobs_entropy_backward(x, None, to_dev(y), None, tau, got[2], got[1], to_dev(g),
                                                        to_dev(gh)))
    _check_grad(d, z, np.ones_like(z), y, tau, g, gh, dtype)


@pytest.mark.parametrize("T,V", [(5, 9001), (800, 2003)], ids=["slices", "whole_rows"])
@pytest.mark.parametrize("tau", [0.7, 1.0, 1.5, 2.0])
@pytest.mark.parametrize("bias", [-1e10, -1e30])
def test_finite_masks_by_bias(T, V, tau, bias):
    """Columns biased out of reach: lanes that hold nothing but touched ones."""
    rng = np.random.default_rng(V + 1)
    x, z = _dev(rng.normal(0, 3, (T, V)), "fp32")
    n = 900
    ids = np.stack([rng.choice(V, n, replace=False) for _ in range(T)])
    ids[0] = np.arange(n)
    y = np.array([rng.choice(np.setdiff1d(np.arange(V), i)) for i in ids])
    z = z.copy()
    np.put_along_axis(z, ids, np.take_along_axis(z, ids, 1) + bias, 1)
    lp = _lp()
    rules = lp.LogitRules(bias_offsets=to_dev(np.arange(T + 1, dtype=np.int64) * n),
                          bias_tokens=to_dev(ids.reshape(-1).astype(np.int32)),
                          bias_values=to_dev(np.full(T * n, bias, dtype=np.float32)))
    got = lp.lp_processed_logprobs_entropy(x, rules, to_dev(y), None, tau)
    _check_scores(got, z, y, tau)
    g, gh = rng.normal(0, 1, T).astype(np.float32), rng.normal(0, 0.5, T).astype(np.float32)
    d = _wide(lp.lp_processed_logprobs_entropy_backward(x, rules, to_dev(y), None, tau, got[2], got[1], to_dev(g),
                                                        to_dev(gh)))
    _check_grad(d, z, np.ones_like(z), y, tau, g, gh, "fp32")


@pytest.mark.parametrize("T,V", [(6, 9001), (800, 2003)], ids=["slices", "whole_rows"])
@pytest.mark.parametrize("value,tau", [(-1e10, 1.0), (-1e10, 1.5), (1e10, 0.7), (-1e30, 1.0), (1e30, 2.0), (-1e38, 0.7),
                                       (1e38, 1.0), (LOWEST["bf16"], 1.5), (LOWEST["bf16"], 2.0), (3e38, 1.0)])
def test_rows_that_are_far_out_as_a_whole(value, tau, T, V):
    """Equal logits share the weight evenly wherever they lie, a single larger
    one takes all of it.  The gradient, whose probabilities come from the fp32
    log-sum-exp, is 0 there."""
    x = np.full((T, V), value, dtype=np.float32)
    x[1::2, V // 3] = np.nextafter(np.float32(value), np.float32(np.inf))
    x[1::2, V // 3] += np.float32(abs(value) * 2.0 ** -20)
    y = np.full(T, 7, dtype=np.int64)
    y[3::4] = V // 3
    lp = _lp()
    xd, yd = to_dev(x), to_dev(y)
    got = lp.lp_processed_logprobs_entropy(xd, None, yd, None, tau)
    a, H, lse = (host(t).astype(np.float64) for t in got)
    assert np.abs(a[0::2] + np.log(V)).max() <= TOL and np.abs(H[0::2] - np.log(V)).max() <= TOL
    assert np.all(H[1::2] == 0) and np.all(a[3::4] == 0)
    gap = (float(x[1, V // 3]) - float(np.float32(value))) / tau
    assert np.all(np.abs(a[1::4] + gap) <= 2.0 ** -21 * gap)
    assert np.all(np.abs(lse - value / tau) <= 2.0 ** -19 * abs(value) / tau)
    one = to_dev(np.ones(T, dtype=np.float32))
    assert not lp.lp_processed_logprobs_entropy_backward(xd, None, yd, None, tau, got[2], got[1], one, one).any()


@pytest.mark.parametrize("T,V", [(6, 9001), (800, 2003)], ids=["slices", "whole_rows"])
@pytest.mark.parametrize("base", [11629080, -11629080, 2000000, -2000000, 16777000 * 3])
def test_neighbouring_whole_numbers(base, T, V):
    """fp32 whole numbers a few apart, on both sides of where exponents are
    taken another way (2^24 / log2(e) = 11629080): their differences count to
    the bit."""
    rng = np.random.default_rng(3)
    step = 4 if abs(base) > 2 ** 24 else 1
    x, z = _dev(np.float32(base) + step * rng.integers(-40, 11, (T, V)), "fp32")
    y = rng.integers(0, V, T).astype(np.int64)
    got = _lp().lp_processed_logprobs_entropy(x, None, to_dev(y), None, 1.0)
    # exponents up to 51 * 4 * log2(e) = 295 of the target, two operations
    want = O.logprobs_entropy(z, y, None, 1.0)
    assert np.abs(host(got[0]) - want[0]).max() <= TOL + 295 * 2.0 ** -23
    assert np.abs(host(got[1]) - want[1]).max() <= TOL
    assert np.all(np.abs(host(got[2]) - want[2]) <= 2.0 ** -22 * np.abs(want[2]))


def test_nan_beside_finite_masks():
    """A NaN shows, wherever it stands among columns out of reach."""
    for T, V in ((6, 9001), (800, 2003)):
        x = np.full((T, V), -1e30, dtype=np.float32)
        x[:, V - 5] = 1.0
        for t in range(0, T, 2):
            x[t, (t * 37) % (V - 5)] = np.nan
        a, H, lse = (host(t) for t in _lp().lp_processed_logprobs_entropy(to_dev(x), None,
                                                                          to_dev(np.full(T, V - 5, dtype=np.int64))))
        for t in (a, H, lse):
            assert np.isnan(t[0::2]).all() and np.isfinite(t[1::2]).all()
        assert np.all(a[1::2] == 0) and np.all(H[1::2] == 0)
