"""GPU parity of the K largest logits against the fp64 oracle: ids equal, log-probs
within tol_log (choose_cases)."""
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


def check(x, z, K, tau=1.0, mask=None):
    """The call on device rows x against the oracle on their fp64 values z."""
    got = [host(g) for g in _lp().lp_top_logits(x, K, None if mask is None else to_dev(mask), tau)]
    with np.errstate(invalid="ignore"):
        want = O.top_logits(z, K, mask, tau)
    assert np.array_equal(got[0], want[0])
    for g, w in zip(got[1:], want[1:]):
        close(g, w, tol_log(w, 2))
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,K", [
    (1, 1, 1), (3, 2, 2), (2, 7, 5), (5, 63, 1), (1, 64, 64), (4, 257, 256), (37, 1000, 17), (2, 2047, 256), (3, 2049, 100),
    (1, 4096, 64), (9, 4097, 20), (2, 20011, 64), (600, 5003, 33), (520, 20011, 64), (515, 20000, 65), (513, 33001, 256),
    (3, 70001, 256), (1, 151936, 20), (2, 131075, 1)])
def test_shapes(dtype, T, V, K):
    rng = np.random.default_rng(T * V + K)
    bits, z = peaked(rng, T, V, dtype, extra=3)
    x = dev_rows(bits, dtype)[:, :V]
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    mask[0] = 1
    check(x, z, K, 0.8, mask)
    y = dev_rows(np.ascontiguousarray(bits[:, :V]), dtype)  # another pitch, and rows off the 16-byte grid
    for a, b in zip(_lp().lp_top_logits(x, K, to_dev(mask), 0.8), _lp().lp_top_logits(y, K, to_dev(mask), 0.8)):
        assert np.array_equal(host(a), host(b))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,K", [(2, 30011, 64), (520, 20011, 50), (517, 20011, 200), (4, 3001, 256), (1, 151936, 256)])
@pytest.mark.parametrize("kind", ["constant", "rising", "falling", "two", "mostly_masked", "mostly_low", "one", "blocks"])
def test_rows_with_no_usable_sample(dtype, T, V, K, kind):
    """Rows whose K-th largest value a sample says nothing of, or that many columns reach."""
    rng = np.random.default_rng(11)
    z = np.zeros((T, V))
    ramp = np.sort(rng.normal(0, 3, V))
    low = {"bf16": -3.3e38, "fp16": -65504.0, "fp32": -3.4e38}[dtype]
    for t in range(T):
        if kind == "constant":
            z[t] = 1.5 - t
        elif kind == "rising":
            z[t] = ramp
        elif kind == "falling":
            z[t] = ramp[::-1]
        elif kind == "two":
            z[t] = rng.integers(0, 2, V)
        elif kind in ("mostly_masked", "mostly_low"):
            z[t] = -np.inf if kind == "mostly_masked" else low
            at = rng.choice(V, min(V, [0, 3, K - 1, K, 5 * K][t % 5]), replace=False)
            z[t, at] = rng.normal(0, 3, at.size)
        elif kind == "one":
            z[t] = -np.inf
            z[t, [V - 1, 0, V // 2][t % 3]] = -2.0
        else:
            z[t] = np.repeat(rng.normal(0, 3, V // 64 + 1), 64)[:V]
    rows = min(T, 9)
    bits = to_bits(z, dtype)
    check(dev_rows(bits, dtype)[:rows], O.widen(bits[:rows], dtype), min(K, V))
    if T > rows:  # a row a workgroup: equal to the sliced rows
        got = _lp().lp_top_logits(dev_rows(bits, dtype), K)
        want = O.top_logits(O.widen(bits[T - 3:], dtype), K, None, 1.0)
        assert np.array_equal(host(got[0])[T - 3:], want[0])
        for g, w in zip(got[1:], want[1:]):
            close(host(g)[T - 3:], w, tol_log(w, 2))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [300, 9001, 40009])
def test_special_values(dtype, V):
    rng = np.random.default_rng(V)
    z = rng.normal(0, 3, (8, V))
    z[0, 7], z[1, V - 1], z[2] = np.nan, np.inf, -np.inf
    z[3, ::2] = -np.inf
    z[4] = np.where(rng.random(V) < 0.5, -0.0, 0.0)  # both zeros are equal: the lowest columns first
    z[5, 5] = z[5, 250] = z[5].max() + 1
    z[6, :40] = -np.inf
    z[7, 100] = np.nan
    z[7, 200] = -np.inf
    bits = to_bits(z, dtype)
    with np.errstate(invalid="ignore"):
        check(dev_rows(bits, dtype), O.widen(bits, dtype), 40, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_extreme_finite_values(dtype):
    """Masks of any size, rows far from zero, and values a type's ulp apart."""
    rng = np.random.default_rng(2)
    V = 5001
    z = rng.normal(0, 3, (6, V))
    z[0, ::3] = -1e4
    if dtype != "fp16":
        z[1, 1::2] = -1e10
        z[2, :4990] = -1e30
    z[3] += 500
    z[4] = 2.0 + rng.integers(0, 9, V) * (2.0 ** -22 if dtype == "fp32" else 2.0 ** -6)
    z[5] -= 3e4
    bits = to_bits(z, dtype)
    check(dev_rows(bits, dtype), O.widen(bits, dtype), 60, 0.7)


def test_outputs_that_are_not_wanted():
    import torch
    z = torch.randn(5, 9000, device="cuda")
    a = _lp().lp_top_logits(z, 9)
    b = _lp().lp_top_logits(z, 9, want_rest=False, want_lse=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and b[2] is None and b[3] is None


def test_empty_and_many_rows():
    import torch
    lp = _lp()
    assert lp.lp_top_logits(torch.zeros(0, 9, device="cuda"), 3)[0].shape == (0, 3)
    T = (1 << 21) + 7003  # more rows than one launch takes
    z = torch.randint(-9, 9, (T, 5), device="cuda").bfloat16()
    ids, p, rest, lse = lp.lp_top_logits(z, 2)
    key = z.float() * 16 - torch.arange(5, device="cuda")
    assert torch.equal(ids, key.topk(2, 1)[1])
    want = torch.log_softmax(z.double(), 1)
    assert (p.double() - want.gather(1, ids)).abs().max() <= 1e-5
    assert (lse.double() - torch.logsumexp(z.double(), 1)).abs().max() <= 1e-5
    left = want.scatter(1, ids, float("-inf"))
    assert (rest.double() - torch.logsumexp(left, 1)).abs().max() <= 1e-5


def test_a_vocabulary_at_the_limit():
    import torch
    V = 1 << 30
    z = torch.zeros(1, V, dtype=torch.bfloat16, device="cuda")
    z[0, V - 1], z[0, 12345678], z[0, V - 2] = 30.0, 20.0, 30.0
    ids, p, rest, lse = _lp().lp_top_logits(z, 4)
    assert ids[0].tolist() == [V - 2, V - 1, 12345678, 0]
    s = 2 * np.exp(30.0) + np.exp(20.0) + V - 3
    close(host(lse), [np.log(s)], 1e-5)
    close(host(rest), [np.log((V - 4) / s)], 1e-5)
    close(host(p)[0], np.array([30, 30, 20, 0]) - np.log(s), 2e-5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,K", [(600, 20011, 3), (600, 20011, 200), (2, 70001, 3)])
def test_rests_and_peaks_anywhere(dtype, T, V, K):
    """The rest far below the list, a rest that lies in a few columns above a far lower floor, values far above the
    first columns', and columns to keep that all lie in one stretch."""
    rng = np.random.default_rng(5)
    z = rng.normal(0, 1, (6, V))
    z[0] -= 150.0
    z[0, rng.choice(V, K, replace=False)] += 150.0       # all else 100 to 200 octaves below
    z[1] -= 300.0
    z[1, rng.choice(V, K + 2, replace=False)] += np.linspace(300, 330, K + 2)
    z[2, V - 5:] += 120.0                                 # the end of the row above all before it
    z[3, V // 2:V // 2 + 700] += np.linspace(3, 9, 700)   # one stretch
    z[4, :K] += np.linspace(200, 100, K)                  # the first columns
    z[5, 1::2] = -np.inf
    bits = to_bits(z, dtype)
    many = np.tile(bits, (T // 6 + 1, 1))[:T]
    x = dev_rows(many, dtype)
    got = [host(g) for g in _lp().lp_top_logits(x, K)]
    rows = min(T, 6)
    want = O.top_logits(O.widen(bits[:rows], dtype), K, None, 1.0)
    assert np.array_equal(got[0][:rows], want[0])
    for g, w in zip(got[1:], want[1:]):
        close(g[:rows], w, tol_log(w, 2))
    for g in got:  # equal rows have equal bits
        assert all(np.array_equal(g[t], g[t % 6]) for t in range(T))


@pytest.mark.parametrize("T,V,K,dtype", [(80, 60740, 22, "fp32"), (68, 135830, 43, "bf16"), (35, 159221, 225, "fp32"),
                                         (51, 60741, 22, "fp32"), (11, 32970, 250, "fp16")])
def test_rows_whose_last_slice_is_shorter(T, V, K, dtype):
    """Slices that are streamed: the last one of a row holds what the others' rounding leaves of it."""
    rng = np.random.default_rng(V)
    bits, z = peaked(rng, T, V, dtype)
    check(dev_rows(bits, dtype), z, K, 1.0)
