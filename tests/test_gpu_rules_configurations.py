"""The calls under rules where rows are many and long: one slice a row of 16384
columns and more, rows that are cut because they are longer than a slice may
be, and more touched columns than are dealt with at a time, against the fp64
oracle on the scored rows (tolerances as in the other tests of these calls)."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.helpers import host, to_dev, to_dev_bits
from tests.rules_cases import EPS, to_bits

pytestmark = pytest.mark.gpu
TOL = 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,V", [(770, 17003), (768, 18000), (770, 170001), (5, 262144)])
def test_long_rows(dtype, T, V):
    import entropy_chunked_row_amd as lp
    rng = np.random.default_rng(T + V)
    n = min(T, 9)
    on = np.sort(rng.choice(T, n, replace=False))
    mask = np.zeros(T, dtype=np.uint8)
    mask[on] = 1
    L, nb = 9000, 1500
    xs = to_bits(rng.normal(0, 3, (n, V)), dtype)
    dev = to_dev if dtype == "fp32" else lambda b: to_dev_bits(b, dtype)
    some = dev(xs)
    x = some.new_full((T, V), 1.0)
    x[to_dev(on)] = some
    tok = rng.integers(-1, V + 1, (2, L)).astype(np.int32)
    hist = rng.integers(0, L + 1, T).astype(np.int32)
    hist[on[:4]] = [0, 1, L, L]
    prompt = (hist // 3).astype(np.int32)
    seq = (np.arange(T) % 2).astype(np.int32)
    rho, f = rng.uniform(0.7, 1.6, T).astype(np.float32), rng.uniform(0, 0.5, T).astype(np.float32)
    off = np.arange(T + 1, dtype=np.int64) * nb
    ids = rng.integers(0, V, T * nb).astype(np.int32)
    val = rng.normal(0, 2, T * nb).astype(np.float32)
    y = rng.integers(0, V, T).astype(np.int64)
    y[on[2]] = tok[seq[on[2]], 0] % V
    words = rng.integers(-2**31, 2**31, (T, (V + 31) // 32)).astype(np.int32)
    words[np.arange(T), y // 32] |= (np.uint32(1) << (y % 32).astype(np.uint32)).view(np.int32)
    rules = lp.LogitRules(tokens=to_dev(tok), hist_len=to_dev(hist), prompt_len=to_dev(prompt), row_seq=to_dev(seq),
                          repetition=to_dev(rho), frequency=to_dev(f), presence=to_dev(f), bias_offsets=to_dev(off),
                          bias_tokens=to_dev(ids), bias_values=to_dev(val), allowed=to_dev(words))
    ok = np.stack([(words[t].view(np.uint32)[:, None] >> np.arange(32, dtype=np.uint32) & 1).reshape(-1)[:V] != 0
                   for t in on])
    z, slope = O.apply_rules(O.widen(xs, dtype), [tok[seq[t], :prompt[t]] for t in on],
                             [tok[seq[t], prompt[t]:hist[t]] for t in on], rho[on], f[on], f[on],
                             [list(zip(ids[off[t]:off[t + 1]], val[off[t]:off[t + 1]])) for t in on], ok)
    md, yd = to_dev(mask), to_dev(y)
    out = x.clone()
    lp.lp_process_logits(x, rules, md, out=out)
    got = host(out[to_dev(on)].float()).astype(np.float64)
    assert np.array_equal(np.isneginf(got), np.isneginf(z))
    fin = np.isfinite(z)
    # six fp32 operations on magnitudes of at most 2 (|z| + 10 counts and a bias), then the type's rounding
    tol = EPS[dtype] / 2 * np.abs(z[fin]) + 6 * 2.0 ** -24 * 2 * (np.abs(O.widen(xs, dtype)[fin]) + 30) + 2.0 ** -25
    assert np.all(np.abs(got[fin] - z[fin]) <= tol)
    off_rows = to_dev(np.nonzero(mask == 0)[0])
    assert bool((out[off_rows] == 1).all())
    tau = 0.8
    a = lp.lp_processed_logprobs_entropy(x, rules, yd, md, tau)
    for p, q in zip(a, O.logprobs_entropy(z, y[on], None, tau)):
        assert np.abs(host(p)[on] - q).max() <= TOL and np.all(host(p)[mask == 0] == 0)
    g, gh = rng.normal(0, 1, T).astype(np.float32), rng.normal(0, 0.5, T).astype(np.float32)
    d = lp.lp_processed_logprobs_entropy_backward(x, rules, yd, md, tau, a[2], a[1], to_dev(g), to_dev(gh))
    want = O.processed_backward(z, slope, y[on], None, tau, g[on], gh[on])
    logp = np.maximum(O.log_softmax(O.tempered(z, tau)), -700)
    size = (np.abs(g) + np.abs(gh))[on, None] * (1 + np.exp(logp) * (np.abs(logp) + 12))
    tol = EPS[dtype] / 2 * np.abs(want) + 2 * TOL * size * np.abs(slope) / tau + 2.0 ** -25
    assert np.all(np.abs(host(d[to_dev(on)].float()) - want) <= tol)
    assert not d[off_rows].any()
    lp.lp_process_logits(x, rules, md, out=x)
    assert bool((x == out).all())
