"""Calls on given logits whose rows hold finite masks: log-prob, entropy and KL
against the fp64 oracle (the bars of the other tests of these calls)."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.helpers import host, to_dev, to_dev_bits
from tests.rules_cases import to_bits

pytestmark = pytest.mark.gpu
TOL = 1e-5
LOWEST = {"bf16": -3.3895313892515355e38, "fp32": -3.4028234663852886e38, "fp16": -65504.0}
MASKS = [("bf16", -1e10), ("bf16", -1e30), ("bf16", -1e38), ("bf16", LOWEST["bf16"]), ("fp32", -1e10), ("fp32", -1e30),
         ("fp32", -1e38), ("fp32", LOWEST["fp32"]), ("fp16", LOWEST["fp16"])]
SIZES = [(12, 1031), (12, 5003), (12, 40009)]


def _dev(x, dtype):
    b = to_bits(x, dtype)
    return (to_dev(b) if dtype == "fp32" else to_dev_bits(b, dtype)), O.widen(b, dtype)


def _kept(T, V, y, rng):
    """Columns that stay, per row: whole lanes and most of a row masked, ahead of what stays and behind it."""
    keep = rng.random((T, V)) < 0.5
    j = np.arange(V)
    keep[0::6], keep[1::6], keep[2::6], keep[3::6] = j >= V - 60, j < 45, j >= V // 2, j // 64 % 2 == 1
    keep[np.arange(T), y] = True
    return keep


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("tau", [0.7, 1.0, 1.5, 2.0])
@pytest.mark.parametrize("dtype,low", MASKS)
def test_logprobs_of_masked_rows(T, V, tau, dtype, low):
    import entropy_chunked_row_amd as lp
    rng = np.random.default_rng(V)
    y = rng.integers(0, V, T).astype(np.int64)
    x, z = _dev(np.where(_kept(T, V, y, rng), rng.normal(0, 3, (T, V)), low), dtype)
    want = O.logprobs_entropy(z, y, None, tau)
    for got, w in zip(lp.lp_logprobs_entropy(x, to_dev(y), None, tau), want):
        assert np.abs(host(got) - w).max() <= TOL
    yk = np.stack([y, y[::-1]], 1)
    k, _ = lp.lp_logprobs_entropy_k(x, to_dev(np.ascontiguousarray(yk)), None, tau)
    assert np.abs(host(k)[:, 0] - want[0]).max() <= TOL


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("value,tau", [(-1e10, 1.0), (-1e10, 0.7), (1e10, 1.5), (-1e30, 1.0), (LOWEST["bf16"], 2.0)])
def test_rows_far_out_as_a_whole(T, V, value, tau):
    import entropy_chunked_row_amd as lp
    x = np.full((T, V), value, dtype=np.float32)
    x[1::2, 5] += np.float32(abs(value) * 2.0 ** -20)
    y = np.full(T, 5, dtype=np.int64)
    a, H = (host(t) for t in lp.lp_logprobs_entropy(to_dev(x), to_dev(y), None, tau))
    assert np.abs(a[0::2] + np.log(V)).max() <= TOL and np.abs(H[0::2] - np.log(V)).max() <= TOL
    assert np.all(a[1::2] == 0) and np.all(H[1::2] == 0)


def test_rows_without_weight_are_nan():
    """Only -inf, or nothing but values whose exponent leaves fp32."""
    import entropy_chunked_row_amd as lp
    for low in (-np.inf, LOWEST["fp32"]):
        x = np.full((4, 5003), low, dtype=np.float32)
        x[1, 17] = 2.0
        a, H = (host(t) for t in lp.lp_logprobs_entropy(to_dev(x), to_dev(np.full(4, 17, dtype=np.int64))))
        assert np.isnan(a[[0, 2, 3]]).all() and np.isnan(H[[0, 2, 3]]).all() and a[1] == 0 and H[1] == 0


@pytest.mark.parametrize("bias", [-1e10, -1e30])
def test_processed_logits_are_scored(bias):
    """A decode step's logits with biases that shut columns out, written and
    then scored as given logits: as scoring under the rules does."""
    import entropy_chunked_row_amd as lp
    rng = np.random.default_rng(5)
    T, V, n = 9, 3001, 1500
    x, z = _dev(rng.normal(0, 3, (T, V)), "fp32")
    ids = np.stack([np.sort(rng.choice(V, n, replace=False)) for _ in range(T)])
    ids[0] = np.arange(n)
    y = np.array([rng.choice(np.setdiff1d(np.arange(V), i)) for i in ids])
    rules = lp.LogitRules(bias_offsets=to_dev(np.arange(T + 1, dtype=np.int64) * n),
                          bias_tokens=to_dev(ids.reshape(-1).astype(np.int32)),
                          bias_values=to_dev(np.full(T * n, bias, dtype=np.float32)))
    z = z.copy()
    np.put_along_axis(z, ids, np.take_along_axis(z, ids, 1) + bias, 1)
    want = O.logprobs_entropy(z, y, None, 0.8)
    got = lp.lp_logprobs_entropy(lp.lp_process_logits(x, rules), to_dev(y), None, 0.8)
    under = lp.lp_processed_logprobs_entropy(x, rules, to_dev(y), None, 0.8)
    for a, b, w in zip(got, under, want):
        assert np.abs(host(a) - w).max() <= TOL and np.abs(host(b) - w).max() <= TOL


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("dtype,low", MASKS)
@pytest.mark.parametrize("subset", [False, True], ids=["same", "subset"])
def test_kl_of_masked_rows(T, V, dtype, low, subset):
    """Both models masked alike, or the teacher more than the student."""
    import entropy_chunked_row_amd as lp
    rng = np.random.default_rng(V + 1)
    y = rng.integers(0, V, T).astype(np.int64)
    keep = _kept(T, V, y, rng)
    u = rng.normal(0, 3, (T, V))
    v = u + rng.normal(0, 0.5, (T, V))
    ut, u64 = _dev(np.where(keep, u, low), dtype)
    only = keep & (rng.random((T, V)) < 0.6) if subset else keep
    only[np.arange(T), y] = True
    vt, v64 = _dev(np.where(only, v, low), dtype)
    got = lp.lp_kl_full_vocab(ut, vt, to_dev(y))
    want = O.kl_and_prob_diff(u64, v64, y, np.ones(T, dtype=np.uint8))
    for g, w in zip(got, want):
        assert np.abs(host(g) - w).max() <= TOL
    # rows off each other's 16-byte grid
    wide = vt.new_empty((T, V + 3))
    wide[:, 1:V + 1] = vt
    for g, w in zip(lp.lp_kl_full_vocab(ut, wide[:, 1:V + 1], to_dev(y)), want):
        assert np.abs(host(g) - w).max() <= TOL
