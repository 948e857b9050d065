"""Rows that finite masks fill: every value as large as a type goes, of either sign.  Values of any size count by how far they
lie below the row's largest, so a row of one value is uniform, and two neighbouring numbers of the type apart are as
far apart as they are.

Log-probs, losses and scores hold to the bounds of ordinary rows (choose_cases); log-sums are as large as the values, and
-inf where fp32 does not hold them."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.choose_cases import SUM, close, dev_rows, tol_log
from tests.helpers import host, to_dev
from tests.rules_cases import DTYPES, to_bits

pytestmark = pytest.mark.gpu
LOW = {"bf16": -3.3895313892515355e38, "fp16": -65504.0, "fp32": float(np.finfo(np.float32).min)}
NEXT = {"bf16": -3.3762390091893825e38, "fp16": -65472.0, "fp32": float(np.nextafter(np.finfo(np.float32).min, np.float32(0)))}


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def _rows(dtype, V):
    """All at the lowest value; one, and every third, at the next one; all at the highest; one ordinary value among
    the lowest; all at -1e30 (fp16: -3e4); ordinary."""
    low, rng = LOW[dtype], np.random.default_rng(V)
    z = np.full((8, V), low)
    z[1, V // 2] = z[2, ::3] = NEXT[dtype]
    z[3] = -low
    z[4, V - 1] = 2.0
    z[5] = -3e4 if dtype == "fp16" else -1e30
    z[6] = rng.normal(0, 2, V)
    z[7, V // 3:V // 3 + 3] = -np.inf
    bits = to_bits(z, dtype)
    return bits, O.widen(bits, dtype)


def _f32(x):
    with np.errstate(over="ignore"):
        return np.asarray(x).astype(np.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [7, 300, 20011, 70001])
@pytest.mark.parametrize("K", [1, 5, 200])
@pytest.mark.parametrize("tau", [1.0, 0.7, 50.0])
def test_top(dtype, V, K, tau):
    tau, K = float(np.float32(tau)), min(K, V)
    bits, z = _rows(dtype, V)
    got = [host(g) for g in _lp().lp_top_logits(dev_rows(bits, dtype), K, None, tau)]
    want = O.top_logits(z, K, None, tau)
    assert np.allclose(want[1][0], -np.log(V)) and np.allclose(want[1][3], -np.log(V))
    assert np.array_equal(got[0], want[0])
    for g, w in zip(got[1:], want[1:]):
        close(g, _f32(w), tol_log(_f32(w), 2))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [9, 300, 20011, 70001])
@pytest.mark.parametrize("tau", [1.0, 0.7, 50.0])
@pytest.mark.parametrize("with_rest", [True, False])
def test_distillation(dtype, V, tau, with_rest):
    tau = float(np.float32(tau))
    bits, z = _rows(dtype, V)
    rng = np.random.default_rng(1)
    ids = np.stack([rng.choice(V, 6, replace=False) for _ in range(8)])
    ids[:, 1] = [V // 2, V // 2, 0, 1, V - 1, 2, 3, V // 3]
    ids[:, 5] = -1
    lpk = np.log(rng.uniform(0.05, 0.2, (8, 6))).astype(np.float32)
    lpk[7, ids[7] == V // 3] = -np.inf
    lpk[4, ids[4] != V - 1] = -1e9  # a teacher under the same mask
    for t in range(8):  # where the student is -inf the teacher has no mass
        lpk[t, (ids[t] >= 0) & np.isneginf(z[t, np.maximum(ids[t], 0)])] = -np.inf
    rest = np.log(rng.uniform(0.05, 0.2, 8)).astype(np.float32) if with_rest else None
    if with_rest:
        rest[4] = -np.inf
    x = dev_rows(bits, dtype)
    args = [to_dev(ids), to_dev(lpk), None if rest is None else to_dev(rest)]
    loss, lse, lse_rest = [host(g) for g in _lp().lp_distill_top(x, *args, None, tau)]
    with np.errstate(over="ignore"):
        want = O.distill_top(z, ids, lpk, rest, None, tau)
    assert np.isfinite(want[0]).all() and np.abs(want[0][[0, 3, 4, 6]]).max() < 40
    close(loss, want[0], 4 * SUM + 2.0 ** -22 * np.abs(want[0]))
    for g, w in ((lse, want[1]), (lse_rest, want[2])):
        close(g, _f32(w), tol_log(_f32(w)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [7, 300, 20011, 70001])
@pytest.mark.parametrize("tau", [1.0, 0.7, 50.0])
def test_beams(dtype, V, tau):
    tau = float(np.float32(tau))
    bits, z = _rows(dtype, V)
    s = np.array([[-0.5, -7.25], [-3.0, -90.0], [-1.0, -55.0], [-2.0, -2.5]], dtype=np.float32)
    z = z[[0, 3, 5, 3, 4, 0, 6, 5]]  # a request: two rows whose scores do not come near each other
    bits = bits[[0, 3, 5, 3, 4, 0, 6, 5]]
    got = [host(g) for g in _lp().lp_beam_select(dev_rows(bits, dtype), to_dev(s), 6, None, 0, tau)]
    want = O.beam_select(z, s, 6, None, 0, tau)
    assert np.isclose(want[0][0, 0], -0.5 - np.log(V))
    for b in range(4):
        if b < 3 or V < 1000:
            assert np.array_equal(got[1][b], want[1][b]) and np.array_equal(got[2][b], want[2][b])
    close(got[0], _f32(want[0]), tol_log(_f32(want[0]), 2))
