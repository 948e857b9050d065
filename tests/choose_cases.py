"""Seeded inputs and tolerances for the calls that choose from rows of logits or distil from what was chosen."""
import numpy as np

from oracle import lp_oracle as O
from tests.rules_cases import EPS, to_bits

# A row's sum of exponentials is off by a relative error of at most 2^-23 (an
# exponential) + 2^-23 |t| (two roundings of its exponent, weighed by its own
# mass: below 4 in all) + 2^-24 for each of at most 130 additions of its chain:
# 1.4e-5 in a log-sum-exp.  Logs and exponents add a few roundings of the value.
SUM = 1.4e-5


def tol_log(ref, sums=1):
    return sums * SUM + 2.0 ** -21 * np.abs(np.where(np.isfinite(ref), ref, 0.0))


def dev_rows(bits, dtype):
    from tests.helpers import to_dev, to_dev_bits
    return to_dev(bits) if dtype == "fp32" else to_dev_bits(bits, dtype)


def close(got, want, tol):
    """Equal where not finite, within tol elsewhere."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True), (got[odd][:5], want[odd][:5])
    err = np.abs(got - want)[~odd]
    lim = np.broadcast_to(np.asarray(tol, dtype=np.float64), want.shape)[~odd]
    assert np.all(err <= lim), (float((err / lim).max()), float(err.max()))


def peaked(rng, T, V, dtype, extra=0):
    """(bits [T, V + extra], fp64 [T, V]): a broad floor and some columns well above it; 16-bit values repeat."""
    z = rng.normal(0, 2, (T, V + extra))
    for t in range(T):
        at = rng.integers(0, V + extra, min(V, 40))
        z[t, at] += rng.uniform(2, 12, at.size)
    bits = to_bits(z, dtype)
    return bits, O.widen(bits, dtype)[:, :V]


def lists(rng, z, K, temperature, pad=True):
    """A teacher's ids, log-probs and log of the rest near rows z: its top, random columns, ids that repeat and ids outside."""
    T, V = z.shape
    v = O.tempered(z + rng.normal(0, 0.5, z.shape), temperature)
    logp = O.log_softmax(v)
    ids = np.zeros((T, K), dtype=np.int64)
    for t in range(T):
        top = np.argsort(-v[t])[:K]
        ids[t] = np.concatenate([top, rng.integers(0, V, K - top.size)])
    lp = np.take_along_axis(logp, ids, 1).astype(np.float32)
    rest = np.full(T, -np.inf)
    for t in range(T):
        left = np.delete(v[t], np.unique(ids[t]))
        if left.size:
            rest[t] = O.log_normaliser(left[None])[0] - O.log_normaliser(v[t:t + 1])[0]
    if pad and K > 3:
        ids[::2, K - 1] = [-1, V, 2**40][T % 3]     # padding
        ids[::3, K - 2] = ids[::3, 0]               # an id twice
        lp[1::2, K - 3] = -np.inf                   # named, without mass
    return ids, lp, rest.astype(np.float32)


def grad_tol(z, ids, lp, rest, temperature, grad_loss, want, dtype):
    """Probabilities are off by a factor of 1 + |lse| 2^-22 + 4 SUM, masses by 2^-22; the result is rounded once."""
    zt = O.tempered(z, temperature)
    tau = temperature if O.temperature_applies(temperature) else 1.0
    tol = np.zeros_like(z)
    for t in range(z.shape[0]):
        at, p, other = O._distill_parts(zt, ids, lp, t)
        p = np.exp(p)
        r = np.exp(float(rest[t])) if rest is not None else 0.0
        lse, lse_rest = O._lse1(zt[t]), O._lse1(zt[t][other])
        part = (p.sum() + r) * np.exp(zt[t] - lse) * (abs(lse) * 2.0 ** -22 + 4 * SUM)
        if np.isfinite(lse_rest):
            part[other] += r * np.exp(zt[t][other] - lse_rest) * ((abs(lse) + abs(lse_rest)) * 2.0 ** -22 + 4 * SUM)
        np.add.at(part, at, p * 2.0 ** -22)
        tol[t] = part * abs(float(grad_loss[t])) / tau
    return tol + EPS[dtype] / 2 * np.abs(want) + (2.0 ** -25 if dtype == "fp16" else 1e-38)
