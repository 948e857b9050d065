"""Rows that spread over more octaves than fp32 has: a reference that a kernel takes early lies far below the row's
largest values, and neither what is left of those nor their sum may be lost.

Row t has its floor g = 60 + 4 t octaves below its few high columns, g up to 320.  Log-sums are compared as everywhere
(choose_cases): exponents are relative to the values that weigh."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.choose_cases import SUM, close, dev_rows, grad_tol, tol_log
from tests.helpers import host, to_dev
from tests.rules_cases import DTYPES, to_bits

pytestmark = pytest.mark.gpu
T = 66


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def _rows(dtype, V, kind, tau=1.0):
    """Row t: high columns at 0, -1, -2 ... times tau, all else near -g.  together: in one vector, at the row's start or
    inside it; apart: one in each 151 columns behind the first two thirds; sorted: up and down, evenly from -2 g on."""
    rng = np.random.default_rng(V)
    z = np.zeros((T, V))
    for t in range(T):
        g = (60 + 4 * t) * np.log(2.0)
        z[t] = -g - rng.random(V)
        if kind == "together":
            at = 0 if t % 2 else (V * 2 // 3) // 8 * 8
            n = min(7, V)
            z[t, at:at + n] = -np.arange(n)[:V - at]
        elif kind == "apart":
            at = np.arange(V * 2 // 3, V, 151)
            z[t, at] = -rng.random(at.size)
            z[t, V - 1] = 0.5
        else:
            z[t] = np.sort(-2 * g * rng.random(V))[::1 if t % 2 else -1]
            z[t] -= z[t].max()
    z *= tau
    bits = to_bits(np.maximum(z, -6e4), dtype)
    return bits, O.widen(bits, dtype)


SHAPES = [13, 900, 12007, 70001]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", SHAPES)
@pytest.mark.parametrize("kind", ["together", "apart", "sorted"])
@pytest.mark.parametrize("tau", [1.0, 0.015625])
def test_top(dtype, V, kind, tau):
    bits, z = _rows(dtype, V, kind, tau)
    x = dev_rows(bits, dtype)
    for K in (1, 2, 5, 100):
        if K > V:
            continue
        for rows in (slice(0, T), slice(20, 22)):  # as many workgroups as rows, or as a row has slices
            got = [host(g) for g in _lp().lp_top_logits(x[rows], K, None, tau)]
            want = O.top_logits(z[rows], K, None, tau)
            assert np.array_equal(got[0], want[0])
            for g, w in zip(got[1:], want[1:]):
                close(g, w, tol_log(w, 2))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", SHAPES)
@pytest.mark.parametrize("kind", ["together", "apart", "sorted"])
def test_beams(dtype, V, kind):
    bits, z = _rows(dtype, V, kind)
    W, N = 3, 4
    s = np.tile(np.array([0.0, -500.0, -1000.0], dtype=np.float32), (T // W, 1))  # beams far apart: no near ties
    got = [host(g) for g in _lp().lp_beam_select(dev_rows(bits, dtype), to_dev(s), N)]
    want = O.beam_select(z, s, N, None, 0, 1.0)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[2], want[2])
    close(got[0], want[0], tol_log(want[0], 2))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", SHAPES)
@pytest.mark.parametrize("kind", ["together", "apart", "sorted"])
@pytest.mark.parametrize("n", [T, 3])
def test_distillation(dtype, V, kind, n):
    """Lists of the largest column, of one high one, or of low ones alone, so that what is left is high or low."""
    bits, z = _rows(dtype, V, kind)
    pick = slice(0, T) if n == T else slice(18, 18 + n)
    bits, z = bits[pick], z[pick]
    top = np.argsort(-z, axis=1, kind="stable")
    ids = np.where((np.arange(n) % 3 == 0)[:, None], top[:, :2], np.where((np.arange(n) % 3 == 1)[:, None], top[:, 1:3], top[:, -2:]))
    lpk = np.tile(np.log(np.array([0.5, 0.2], dtype=np.float32)), (n, 1))
    rest = np.full(n, np.log(0.3), dtype=np.float32)
    x, a = dev_rows(bits, dtype), [to_dev(t) for t in (ids, lpk, rest)]
    got = _lp().lp_distill_top(x, *a)
    want = O.distill_top(z, ids, lpk, rest, None, 1.0)
    close(host(got[0]), want[0], 4 * SUM + 2.0 ** -22 * np.abs(want[0]))
    for g, w in zip(got[1:], want[1:]):
        close(host(g), w, tol_log(w))
    gl = np.ones(n, dtype=np.float32)
    d = _lp().lp_distill_top_backward(x, *a, None, 1.0, got[1], got[2], to_dev(gl))
    ref = O.distill_top_backward(z, ids, lpk, rest, None, 1.0, gl)
    # probabilities below 2^-126 may be flushed
    close(host(d.float()), ref, grad_tol(z, ids, lpk, rest, 1.0, gl, ref, dtype) + 2.0 ** -125)
