"""GPU parity of the calls under logit rules against the fp64 oracle.

Tolerances, derived before the first run.
* process: at most six fp32 operations of relative error 2^-24 on values no
  larger than M = 2 (|z| + |f| n + |p| + |b|) (rho is within 0.7 .. 1.6), then
  one rounding to the type, eps / 2 relative: eps/2 |z| + 6 * 2^-24 M, plus half
  the smallest subnormal of fp16 (2^-25).
* score: the bar of the other logits calls, 1e-5 absolute: exponents up to
  |z| / tau log2(e) <= 64 carry 64 * 2^-24 = 4e-6.
* gradient: a probability's relative error is that of its exponent, 1e-5 by
  the same count (the rounded lse doubles it), on a sum of terms
  (|g| + |gH| (|log p| + H)) p slope / tau; then the type's rounding as above."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.helpers import host, to_dev, to_dev_bits
from tests.rules_cases import DTYPES, EPS, Rules, to_bits

pytestmark = pytest.mark.gpu
TOL = 1e-5


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def _torch():
    import torch
    return torch


def _wide(t):
    return host(t.float()).astype(np.float64)


def _same_or_near(got, want, tol):
    """Equal where `want` is not finite, within `tol` elsewhere."""
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    err = np.abs(got[fin] - want[fin])
    assert np.all(err <= np.broadcast_to(tol, want.shape)[fin]), float((err - np.broadcast_to(tol, want.shape)[fin]).max())


def _process_tol(c, z):
    n = c.tokens.shape[1] if hasattr(c, "tokens") else 0
    M = 2 * (np.abs(c.logits64()) + n + 1 + 10)
    with np.errstate(invalid="ignore"):
        return EPS[c.dtype] / 2 * np.abs(z) + 6 * 2.0 ** -24 * M + 2.0 ** -25


CASES = [dict(), dict(shared=True), dict(history=False), dict(bias=False), dict(grammar=False),
         dict(history=False, bias=False, grammar=False), dict(extra_cols=3, extra_len=5), dict(extra_cols=8)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 8, 31, 33, 1000, 1031, 4097, 9001])
@pytest.mark.parametrize("kw", CASES, ids=lambda k: "-".join(k) or "all")
def test_process(dtype, V, kw):
    torch = _torch()
    c = Rules(7, V, dtype, seed=V, **kw)
    x, rules = c.device()
    z, _ = c.processed()
    before = x.clone()
    got = _wide(_lp().lp_process_logits(x, rules))
    _same_or_near(got, z, _process_tol(c, z))
    assert torch.equal(x, before)
    # rows of mask 0 keep what out held; so does everything past V
    out = torch.full((7, V + 5), 123.0, dtype=x.dtype, device="cuda")
    _lp().lp_process_logits(x, rules, to_dev(c.mask), out=out[:, 2:2 + V])
    o = _wide(out)
    assert np.all(o[:, :2] == 123) and np.all(o[:, 2 + V:] == 123) and np.all(o[c.mask == 0] == 123)
    assert np.array_equal(o[c.mask != 0, 2:2 + V], got[c.mask != 0], equal_nan=True)
    # in place
    _lp().lp_process_logits(x, rules, to_dev(c.mask), out=x)
    xi = _wide(x)
    assert np.array_equal(xi[c.mask != 0], got[c.mask != 0], equal_nan=True)
    assert np.array_equal(xi[c.mask == 0], _wide(before)[c.mask == 0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_special_values_under_the_grammar(dtype):
    """NaN and +-inf in columns that are not allowed do not show; the type's
    lowest value and -inf in allowed ones weigh nothing."""
    c = Rules(9, 501, dtype, seed=3, history=False, bias=False).plant_specials()
    x, rules = c.device()
    z, slope = c.processed()
    _same_or_near(_wide(_lp().lp_process_logits(x, rules)), z, 2.0 ** -24 * 0 + EPS[dtype] / 2 * np.abs(z, where=np.isfinite(z), out=np.zeros_like(z)))
    y = to_dev(c.targets)
    lp_g, H_g, lse_g = _lp().lp_processed_logprobs_entropy(x, rules, y, None, 0.7)
    keep = [t for t in range(9) if t != 4]
    lp_o, H_o, _ = O.logprobs_entropy(z[keep], c.targets[keep], None, 0.7)
    assert np.abs(host(lp_g)[keep] - lp_o).max() <= TOL and np.abs(host(H_g)[keep] - H_o).max() <= TOL
    # row 4 allows nothing
    assert np.isnan(host(lp_g)[4]) and np.isnan(host(H_g)[4]) and host(lse_g)[4] == -np.inf
    g, gh = np.linspace(-1, 1, 9).astype(np.float32), np.linspace(0.5, -0.5, 9).astype(np.float32)
    d = _wide(_lp().lp_processed_logprobs_entropy_backward(x, rules, y, None, 0.7, lse_g, H_g, to_dev(g), to_dev(gh)))
    assert np.all(np.isfinite(d)) and np.all(d[4] == 0) and np.all(d[~c.oracle["allowed"]] == 0)
    want = O.processed_backward(z, slope, c.targets, None, 0.7, g, gh)
    assert np.abs(d - want).max() <= EPS[dtype] / 2 * 2 + 1e-4


def test_nan_and_inf_rows():
    """A row whose allowed logits hold a NaN or +inf is NaN, its neighbours are not touched."""
    torch = _torch()
    x = torch.zeros(4, 3000, device="cuda")
    x[1, 2999] = float("nan")
    x[2, 5] = float("inf")
    y = torch.zeros(4, dtype=torch.int64, device="cuda")
    out = [host(t) for t in _lp().lp_processed_logprobs_entropy(x, None, y, None, 1.0)]
    for t in out[:2]:
        assert np.isnan(t[1]) and np.isnan(t[2]) and np.isfinite(t[[0, 3]]).all()
    x[0, :] = -float("inf")
    lp_g, H_g, lse_g = [host(t) for t in _lp().lp_processed_logprobs_entropy(x, None, y, None, 1.0)]
    assert np.isnan(lp_g[0]) and np.isnan(H_g[0]) and lse_g[0] == -np.inf and abs(lse_g[3] - np.log(3000)) <= TOL


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 8, 31, 33, 1000, 1031, 4097, 9001])
@pytest.mark.parametrize("kw,tau", [(dict(), 0.7), (dict(shared=True, extra_cols=3), 1.0), (dict(history=False), 1.4),
                                    (dict(bias=False, extra_len=3), 0.7), (dict(grammar=False), 0.7)],
                         ids=["all", "shared", "no_history", "no_bias", "no_grammar"])
def test_score_and_gradient(dtype, V, kw, tau):
    c = Rules(11, V, dtype, seed=V + 1, empty_row=False, **kw)
    x, rules = c.device()
    z, slope = c.processed()
    y, m = to_dev(c.targets), to_dev(c.mask)
    lp_g, H_g, lse_g = _lp().lp_processed_logprobs_entropy(x, rules, y, m, tau)
    lp_o, H_o, lse_o = O.logprobs_entropy(z, c.targets, c.mask, tau)
    on = c.mask != 0
    for got, want in ((lp_g, lp_o), (H_g, H_o)):
        assert np.abs(host(got) - want).max() <= TOL
        assert np.all(host(got)[~on] == 0)
    assert np.abs(host(lse_g)[on] - np.asarray(lse_o)[on]).max() <= TOL
    rng = np.random.default_rng(V)
    g = rng.normal(0, 1, 11).astype(np.float32)
    gh = rng.normal(0, 0.5, 11).astype(np.float32)
    for ent in (gh, None):
        d = _wide(_lp().lp_processed_logprobs_entropy_backward(x, rules, y, m, tau, lse_g, H_g, to_dev(g),
                                                               None if ent is None else to_dev(ent)))
        want = O.processed_backward(z, slope, c.targets, c.mask, tau, g, ent)
        with np.errstate(divide="ignore"):
            logp = np.log(np.maximum(np.exp(O.log_softmax(O.tempered(z, tau))), 1e-300))
        size = (np.abs(g) + (0 if ent is None else np.abs(ent)))[:, None] * (1 + np.exp(logp) * (np.abs(logp) + 12))
        _same_or_near(d, want, EPS[dtype] / 2 * np.abs(want) + 2 * TOL * size * np.abs(slope) / tau + 2.0 ** -25)
        assert np.all(d[~on] == 0)


def test_no_rules_is_the_plain_call():
    c = Rules(16, 5003, "bf16", seed=2)
    x, _ = c.device()
    y, m = to_dev(c.targets), to_dev(c.mask)
    a = [host(t) for t in _lp().lp_processed_logprobs_entropy(x, None, y, m, 0.7)[:2]]
    b = [host(t) for t in _lp().lp_logprobs_entropy(x, y, m, 0.7)]
    assert all(np.abs(p - q).max() <= TOL for p, q in zip(a, b))


def test_targets_out_of_range_and_not_allowed():
    torch = _torch()
    V = 100
    x = torch.zeros(4, V, dtype=torch.bfloat16, device="cuda")
    y = to_dev(np.array([V, -1, 3, 64], dtype=np.int64))
    words = torch.full((4, 4), -1, dtype=torch.int32, device="cuda")
    words[2, 0] = ~(1 << 3)
    lp_g, H_g, lse = _lp().lp_processed_logprobs_entropy(x, _lp().LogitRules(allowed=words), y)
    lp_g, H_g = host(lp_g), host(H_g)
    assert np.isnan(lp_g[:2]).all() and lp_g[2] == -np.inf and abs(lp_g[3] + np.log(V)) <= TOL
    assert np.abs(H_g - np.log([V, V, V - 1, V])).max() <= TOL
    g = torch.ones(4, device="cuda")
    d = _wide(_lp().lp_processed_logprobs_entropy_backward(x, _lp().LogitRules(allowed=words), y, None, 1.0, lse,
                                                           to_dev(H_g), g))
    assert np.abs(d[:2] + 1 / V).max() <= 1e-4 and d[2, 3] == 0 and abs(d[2, 4] + 1 / (V - 1)) <= 1e-4
    assert abs(d[3, 64] - (1 - 1 / V)) <= 4e-3


def test_bad_indices_in_device_arrays_stay_in_bounds():
    """Lengths, buffer indices and offsets beyond their arrays are clamped."""
    torch = _torch()
    lp = _lp()
    V, L = 50, 8
    x = torch.randn(4, V, device="cuda")
    tok = torch.arange(3 * L, device="cuda", dtype=torch.int32).view(3, L) % V
    one = torch.ones(4, device="cuda")
    r = lp.LogitRules(tokens=tok, hist_len=to_dev(np.array([2**31 - 1, -5, L + 1, 3], dtype=np.int32)),
                      prompt_len=to_dev(np.array([-7, 3, 2**31 - 1, 0], dtype=np.int32)),
                      row_seq=to_dev(np.array([0, 1, 2, 3], dtype=np.int32)), presence=one,
                      bias_offsets=to_dev(np.array([-4, 2**60, 1, 0, -2**60], dtype=np.int64)),
                      bias_tokens=to_dev(np.array([7, 9], dtype=np.int32)), bias_values=to_dev(np.array([4, 8], dtype=np.float32)))
    z, _ = O.apply_rules(host(x), [[], [], range(2 * L, 3 * L), []], [range(L), [], [], []], presence=host(one),
                         biases=[[(7, 4), (9, 8)], [], [], []])
    got = host(lp.lp_process_logits(x, r))
    assert np.abs(got - z).max() <= 1e-5


def test_counts_are_exact_over_long_histories():
    """One token ten thousand times, over several rows of one buffer."""
    torch = _torch()
    lp = _lp()
    V, L = 3001, 20000
    tok = torch.full((1, L), 2777, dtype=torch.int32, device="cuda")
    tok[0, 1::2] = torch.arange(L // 2, device="cuda", dtype=torch.int32) % V
    x = torch.zeros(3, V, device="cuda")
    lens = [0, 1, L]
    r = lp.LogitRules(tokens=tok, hist_len=to_dev(np.array(lens, dtype=np.int32)), row_seq=torch.zeros(3, dtype=torch.int32, device="cuda"),
                      frequency=torch.ones(3, device="cuda"))
    got = host(lp.lp_process_logits(x, r))
    th = host(tok)[0]
    for row, n in enumerate(lens):
        assert np.array_equal(-got[row], np.bincount(th[:n], minlength=V).astype(np.float32))


def test_empty_batches():
    torch = _torch()
    lp = _lp()
    x = torch.zeros((0, 100), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(0, dtype=torch.int64, device="cuda")
    f = torch.zeros(0, device="cuda")
    r = lp.LogitRules(tokens=torch.zeros((0, 5), dtype=torch.int32, device="cuda"), hist_len=y.int(), presence=f,
                      bias_offsets=torch.zeros(1, dtype=torch.int64, device="cuda"), bias_tokens=y.int(), bias_values=f,
                      allowed=torch.zeros((0, 4), dtype=torch.int32, device="cuda"))
    assert lp.lp_process_logits(x, r).shape == (0, 100)
    assert all(t.numel() == 0 for t in lp.lp_processed_logprobs_entropy(x, r, y))
    assert lp.lp_processed_logprobs_entropy_backward(x, r, y, None, 1.0, f, f, f, f).shape == (0, 100)
    # rows without any buffered token
    x1 = torch.ones((1, 100), device="cuda")
    r = lp.LogitRules(tokens=torch.zeros((1, 0), dtype=torch.int32, device="cuda"),
                      hist_len=torch.zeros(1, dtype=torch.int32, device="cuda"), presence=torch.ones(1, device="cuda"))
    assert torch.equal(lp.lp_process_logits(x1, r), x1)


def test_offsets_past_32_bits():
    """A row more than 2^32 bytes into the logits, the mask and the output."""
    torch = _torch()
    lp = _lp()
    V, T = 65536, 33000  # 2.16e9 elements
    c = Rules(1, V, "bf16", seed=8)
    xr, rules = c.device()
    x = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    x[-1] = xr[0]
    want = lp.lp_process_logits(xr, rules)
    y = torch.full((T,), int(c.targets[0]), dtype=torch.int64, device="cuda")
    allowed = torch.full((T, V // 32), -1, dtype=torch.int32, device="cuda")
    allowed[-1] = to_dev(c.args["allowed"])[0]
    hist = torch.zeros(T, dtype=torch.int32, device="cuda")
    hist[-1] = int(c.args["hist_len"][0])
    pr = torch.full((T,), int(c.args["prompt_len"][0]), dtype=torch.int32, device="cuda")
    full = lambda k: torch.full((T,), float(c.args[k][0]), device="cuda")  # noqa: E731
    off = torch.zeros(T + 1, dtype=torch.int64, device="cuda")
    off[-1] = int(c.args["bias_offsets"][-1])
    r = lp.LogitRules(tokens=to_dev(c.tokens), hist_len=hist, prompt_len=pr,
                      row_seq=torch.zeros(T, dtype=torch.int32, device="cuda"), repetition=full("repetition"),
                      frequency=full("frequency"), presence=full("presence"), bias_offsets=off,
                      bias_tokens=to_dev(c.args["bias_tokens"]), bias_values=to_dev(c.args["bias_values"]),
                      allowed=allowed)
    m = torch.zeros(T, dtype=torch.uint8, device="cuda")
    m[-1] = 1
    out = torch.zeros_like(x)
    lp.lp_process_logits(x, r, m, out=out)
    assert torch.equal(out[-1], want[0]) and not out[:-1].any()
    a = lp.lp_processed_logprobs_entropy(x, r, y, m, 0.7)
    b = lp.lp_processed_logprobs_entropy(xr, rules, y[-1:], None, 0.7)
    assert all(abs(float(p[-1]) - float(q[0])) <= TOL for p, q in zip(a, b))
    g = torch.ones(T, device="cuda")
    lp.lp_processed_logprobs_entropy_backward(x, r, y, m, 0.7, a[2], a[1], g, g, grad_logits=out)
    d = lp.lp_processed_logprobs_entropy_backward(xr, rules, y[-1:], None, 0.7, a[2][-1:], a[1][-1:], g[:1], g[:1])
    assert torch.equal(out[-1], d[0]) and not out[:-1].any()


def test_captured_and_on_another_stream():
    """A decode step captured into a graph (process, score, gradient) replays
    on new inputs; the same calls on a side stream agree bit for bit."""
    torch = _torch()
    lp = _lp()
    cs = [Rules(5, 9001, "fp16", seed=s, empty_row=False) for s in (1, 2, 3)]
    first, rules = cs[0].device()
    x = first.clone()
    kept = {n: t for n, t in rules._whole + rules._per_row}
    y = to_dev(cs[0].targets)
    g = torch.linspace(-1, 1, 5, device="cuda")

    def step(stream=None):
        z = lp.lp_process_logits(x, rules, stream=stream)
        a = lp.lp_processed_logprobs_entropy(x, rules, y, None, 0.7, stream=stream)
        d = lp.lp_processed_logprobs_entropy_backward(x, rules, y, None, 0.7, a[2], a[1], g, g, stream=stream)
        return [z, *a, d]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    side = torch.cuda.Stream()
    for k in range(6):
        c = cs[k % 3]
        x.copy_(c.device()[0])
        y.copy_(to_dev(c.targets))
        kept["hist_len"].copy_(to_dev(c.args["hist_len"]).clamp(max=kept["tokens"].shape[1]))
        kept["allowed"].copy_(to_dev(c.args["allowed"]))
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, eager)), k
        other = step(side)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(other, eager)), k


def test_repeatable_bit_for_bit():
    torch = _torch()
    lp = _lp()
    c = Rules(40, 20011, "bf16", seed=6, L=400)
    x, rules = c.device()
    y = to_dev(c.targets)
    a = lp.lp_processed_logprobs_entropy(x, rules, y, None, 0.7)
    for _ in range(3):
        b = lp.lp_processed_logprobs_entropy(x, rules, y, None, 0.7)
        assert all(torch.equal(p.view(torch.int32), q.view(torch.int32)) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_touched_columns_in_many_rows(dtype):
    """Rows enough for one workgroup a row, whose histories and biases touch
    most of the vocabulary: more columns than are dealt with at a time."""
    torch = _torch()
    lp = _lp()
    rng = np.random.default_rng(12)
    T, V, L = 1100, 9001, 12000
    bits = to_bits(rng.normal(0, 3, (T, V)), dtype)
    tok = rng.integers(0, V, (2, L)).astype(np.int32)
    seq = (np.arange(T) % 2).astype(np.int32)
    hist = rng.integers(0, L + 1, T).astype(np.int32)
    hist[5:8] = [0, 1, L]
    prompt = (hist // 3).astype(np.int32)
    nb = rng.choice([0, 1, 40], T)
    nb[6] = 5000
    off = np.concatenate([[0], np.cumsum(nb)]).astype(np.int64)
    ids = rng.integers(0, V, off[-1]).astype(np.int32)
    val = rng.normal(0, 2, off[-1]).astype(np.float32)
    rho, f = rng.uniform(0.7, 1.6, T).astype(np.float32), rng.uniform(0, 0.5, T).astype(np.float32)
    words = rng.integers(-2**31, 2**31, (T, (V + 31) // 32)).astype(np.int32)
    x = to_dev(bits) if dtype == "fp32" else to_dev_bits(bits, dtype)
    y = rng.integers(0, V, T).astype(np.int64)
    words[np.arange(T), y // 32] |= (np.uint32(1) << (y % 32).astype(np.uint32)).view(np.int32)
    r = lp.LogitRules(tokens=to_dev(tok), hist_len=to_dev(hist), prompt_len=to_dev(prompt), row_seq=to_dev(seq),
                      repetition=to_dev(rho), frequency=to_dev(f), presence=to_dev(f), bias_offsets=to_dev(off),
                      bias_tokens=to_dev(ids), bias_values=to_dev(val), allowed=to_dev(words))
    z = O.widen(bits, dtype)
    slope = np.ones((T, V))
    mag = np.abs(z)
    for t in range(T):
        h = tok[seq[t], :hist[t]]
        times = np.bincount(h[prompt[t]:], minlength=V)
        seen = np.bincount(h, minlength=V) > 0
        slope[t, seen] = np.where(z[t, seen] > 0, 1 / float(rho[t]), float(rho[t]))
        z[t] = z[t] * slope[t] - float(f[t]) * (times + (times > 0))
        mag[t] = 2 * mag[t] + np.abs(float(f[t])) * (times + 1)
        for j, b in {int(i): float(v) for i, v in zip(ids[off[t]:off[t + 1]], val[off[t]:off[t + 1]])}.items():
            z[t, j] += b
            mag[t, j] += abs(b)
        ok = (words[t].view(np.uint32)[:, None] >> np.arange(32, dtype=np.uint32) & 1).reshape(-1)[:V] != 0
        z[t, ~ok] = -np.inf
        slope[t, ~ok] = 0
    got = _wide(lp.lp_process_logits(x, r))
    zf = np.where(np.isfinite(z), z, 0)
    _same_or_near(got, z, EPS[dtype] / 2 * np.abs(zf) + 6 * 2.0 ** -24 * mag + 2.0 ** -25)
    yd = to_dev(y)
    a = lp.lp_processed_logprobs_entropy(x, r, yd, None, 0.9)
    lp_o, H_o, lse_o = O.logprobs_entropy(z, y, None, 0.9)
    for p, q in zip(a, (lp_o, H_o, lse_o)):
        assert np.abs(host(p) - q).max() <= TOL
    g = rng.normal(0, 1, T).astype(np.float32)
    d = _wide(lp.lp_processed_logprobs_entropy_backward(x, r, yd, None, 0.9, a[2], a[1], to_dev(g), to_dev(f)))
    want = O.processed_backward(z, slope, y, None, 0.9, g, f)
    assert np.all(np.abs(d - want) <= EPS[dtype] / 2 * np.abs(want) + 2 * TOL * (np.abs(g) + f * 30)[:, None] * 1.6 + 2.0 ** -25)
    lp.lp_process_logits(x, r, out=x)
    assert np.array_equal(_wide(x), got)


def test_inputs_unchanged_and_two_streams_at_once():
    """No call writes its inputs (the logits processed in place apart), and
    calls that overlap on two streams agree with the calls made alone."""
    torch = _torch()
    lp = _lp()
    cs = [Rules(300, 5003, "bf16", seed=s, L=500, empty_row=False) for s in (31, 32)]
    dv = [c.device() for c in cs]
    ys = [to_dev(c.targets) for c in cs]
    g = torch.linspace(-1, 1, 300, device="cuda")
    inputs = [t for x, r in dv for t in (x, *(v for _, v in r._whole + r._per_row))] + ys + [g]
    kept = [t.clone() for t in inputs]

    def step(k, stream=None):
        (x, r), y = dv[k], ys[k]
        a = lp.lp_processed_logprobs_entropy(x, r, y, None, 0.7, stream=stream)
        d = lp.lp_processed_logprobs_entropy_backward(x, r, y, None, 0.7, a[2], a[1], g, g, stream=stream)
        return [lp.lp_process_logits(x, r, stream=stream), *a, d]

    alone = [step(k) for k in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [step(k, streams[k]) for k in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for p, q in zip(got, alone) for a, b in zip(p, q))
    assert all(torch.equal(a, b) for a, b in zip(kept, inputs))


def test_temperatures_that_do_not_apply():
    """tau <= 0 and tau == 1 leave the logits as they are, in both directions."""
    torch = _torch()
    lp = _lp()
    c = Rules(6, 300, "fp32", seed=9, empty_row=False)
    x, r = c.device()
    y, g = to_dev(c.targets), torch.ones(6, device="cuda")
    base = lp.lp_processed_logprobs_entropy(x, r, y, None, 1.0)
    d = lp.lp_processed_logprobs_entropy_backward(x, r, y, None, 1.0, base[2], base[1], g, g)
    for tau in (0.0, -2.0):
        a = lp.lp_processed_logprobs_entropy(x, r, y, None, tau)
        assert all(torch.equal(p, q) for p, q in zip(a, base))
        assert torch.equal(lp.lp_processed_logprobs_entropy_backward(x, r, y, None, tau, a[2], a[1], g, g), d)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_the_types_lowest_value(dtype):
    """Allowed logits that all hold the lowest fp16 share the weight evenly:
    what the grammar shuts out stays out.  The lowest bf16 and fp32 weigh nothing:
    rows of them are NaN with lse -inf, and have no gradient."""
    torch = _torch()
    lp = _lp()
    t = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dtype]
    V = 2000
    x = torch.full((2, V), torch.finfo(t).min, dtype=t, device="cuda")
    x[1, :1000] = 0  # not allowed, and far above the others
    words = torch.full((2, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    words[1, :1000 // 32] = 0
    words[1, 1000 // 32] = -1 << (1000 % 32)
    y = torch.tensor([5, 1500], device="cuda")
    rules = lp.LogitRules(allowed=words)
    lp_g, H_g, lse_g = lp.lp_processed_logprobs_entropy(x, rules, y)
    g = torch.ones(2, device="cuda")
    d = _wide(lp.lp_processed_logprobs_entropy_backward(x, rules, y, None, 1.0, lse_g, H_g, g, g))
    if dtype == "fp16":
        n = np.array([V, 1000])
        assert np.abs(host(lp_g) + np.log(n)).max() <= TOL and np.abs(host(H_g) - np.log(n)).max() <= TOL
        # log2 p carries roundings at 94502 = 65504 log2(e): of mc + log2 s and of lse log2(e), 2^-8 each, of lse
        # itself, 2^-9 log2(e), and of the product of the rounded ln 2 and log2(e), 94502 2^-24: 0.0163 together,
        # so p by 1.14 %, and the entropy's p (log p + H) by 1.14 % of p; 2^-5 covers both.
        want = np.zeros((2, V))
        want[0], want[1, 1000:] = -1 / n[0], -1 / n[1]
        want[0, 5] += 1
        want[1, 1500] += 1
        assert np.all(np.abs(d - want) <= np.abs(want) * 2.0 ** -11 + 1e-3 * 2 ** -5)
    else:
        assert np.all(np.isnan(host(lp_g))) and np.all(np.isnan(host(H_g))) and np.all(host(lse_g) == -np.inf)
        assert np.all(d == 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [70001, 70016])
def test_process_slices_of_long_rows(dtype, V):
    """Rows in four slices each, of many vectors a lane, in place too."""
    c = Rules(200, V, dtype, seed=V, L=700)
    x, rules = c.device()
    z, _ = c.processed()
    got = _wide(_lp().lp_process_logits(x, rules))
    _same_or_near(got, z, _process_tol(c, z))
    _lp().lp_process_logits(x, rules, out=x)
    assert np.array_equal(_wide(x), got, equal_nan=True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_logits_of_a_padded_vocabulary(dtype):
    """Rows of the logits and of what is written start on different boundaries."""
    c = Rules(21, 9001, dtype, seed=77, extra_cols=15, empty_row=False)
    x, rules = c.device()
    z, slope = c.processed()
    got = _wide(_lp().lp_process_logits(x, rules))
    _same_or_near(got, z, _process_tol(c, z))
    y = to_dev(c.targets)
    args = (rules, y, None, 0.7)
    lp_g, H_g, lse_g = _lp().lp_processed_logprobs_entropy(x, *args)
    g = to_dev(np.linspace(-1, 1, 21).astype(np.float32))
    d = _lp().lp_processed_logprobs_entropy_backward(x, *args, lse_g, H_g, g, g)
    same = x.contiguous()
    assert np.array_equal(_wide(_lp().lp_process_logits(same, rules)), got, equal_nan=True)
    assert np.abs(host(lp_g) - O.logprobs_entropy(z, c.targets, None, 0.7)[0]).max() <= TOL
    # the same lse, so the same gradient to the bit, whatever the rows' boundaries
    assert _torch().equal(_lp().lp_processed_logprobs_entropy_backward(same, *args, lse_g, H_g, g, g), d)
