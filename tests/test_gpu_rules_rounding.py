"""The rules are fp32 operations each rounded on its own: fp32 results equal
numpy's step by step, to the bit."""
import numpy as np
import pytest

from tests.helpers import host, to_dev, to_dev_bits
from tests.rules_cases import to_bits

pytestmark = pytest.mark.gpu


def _steps(x, seen, times, rho, f, p, bias):
    """The formula in numpy fp32, an operation at a time."""
    x = x.astype(np.float32)
    z = np.where(seen, np.where(x > 0, x / rho, x * rho), x)
    out = times > 0
    z = np.where(out, z - f * times.astype(np.float32), z)
    z = np.where(out, z - p, z)
    return np.where(np.isnan(bias), z, z + bias).astype(np.float32)


@pytest.mark.parametrize("T,V", [(7, 1031), (9, 20011), (800, 5003)])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_every_step_is_rounded(T, V, seed):
    import torch

    import entropy_chunked_row_amd as lp
    rng = np.random.default_rng(seed)
    L = 300
    x = rng.normal(0, 3, (T, V)).astype(np.float32)
    pool = rng.integers(0, V, 40)
    tok = rng.choice(pool, (T, L)).astype(np.int32)
    hist = rng.integers(L // 2, L + 1, T)
    prompt = rng.integers(0, L // 2, T)
    # no product of a penalty with a count is a 24-bit number
    rho, f, p = (rng.uniform(lo, hi, (T, 1)).astype(np.float32) for lo, hi in ((0.7, 1.6), (0.1, 1.0), (0.1, 1.0)))
    nb = 12
    ids = np.stack([np.concatenate([rng.choice(np.unique(tok[t]), 6, replace=False),
                                    rng.choice(np.setdiff1d(np.arange(V), pool), 6, replace=False)]) for t in range(T)])
    val = rng.normal(0, 2, (T, nb)).astype(np.float32)
    seen, times, bias = np.zeros((T, V), bool), np.zeros((T, V), np.int64), np.full((T, V), np.nan, np.float32)
    for t in range(T):
        seen[t, tok[t, :hist[t]]] = True
        times[t] = np.bincount(tok[t, prompt[t]:hist[t]], minlength=V)
        bias[t, ids[t]] = val[t]
    rules = lp.LogitRules(tokens=to_dev(tok), hist_len=to_dev(hist.astype(np.int32)),
                          prompt_len=to_dev(prompt.astype(np.int32)), repetition=to_dev(rho[:, 0]),
                          frequency=to_dev(f[:, 0]), presence=to_dev(p[:, 0]),
                          bias_offsets=to_dev(np.arange(T + 1, dtype=np.int64) * nb),
                          bias_tokens=to_dev(ids.reshape(-1).astype(np.int32)), bias_values=to_dev(val.reshape(-1)))
    want = _steps(x, seen, times, rho, f, p, bias)
    got = host(lp.lp_process_logits(to_dev(x), rules))
    assert np.array_equal(got.view(np.uint32), want.view(np.uint32))
    # 16-bit logits: the same steps on the widened values, rounded once at the end
    for dtype in ("bf16", "fp16"):
        b = to_bits(x, dtype)
        wide = host(to_dev_bits(b, dtype).float())
        want = to_bits(_steps(wide, seen, times, rho, f, p, bias), dtype)
        out = lp.lp_process_logits(to_dev_bits(b, dtype), rules)
        assert np.array_equal(host(out.view(torch.int16)).view(np.uint16), want)
