"""How exactly the 8-bit head sums.

Sums of one product each are exact in every kernel.  For 16-bit results of more than 16 rows (of any number past h = 8192)
the 8-bit instructions drop what lies 2^-13 below the largest of 8 products: each loses less than u = 2^-13 of that one,
with its own sign, u / sqrt(3) of rms where what is lost is spread evenly.  The square of the largest of 8 is at most the
sum of their squares, so over h products of rms r, whose sum has rms r sqrt(h), the errors have an rms below
2^-13 sqrt(8 / 3) = 2.0e-4 of the logits'.  Sums that cancel show it alone: their results are as small as the error, so that
rounding them to 16 bits adds EPS / 2 of it."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.helpers import host, to_dev_bits
from tests.rules_cases import EPS, to_bits

pytestmark = pytest.mark.gpu
OUT = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def _torch():
    import torch
    return torch


@pytest.mark.parametrize("out", ["bf16", "fp16"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 16, 17, 32, 33, 64, 65, 128, 129, 300])
def test_sums_of_one_product_are_exact(out, dtype, T):
    """Through a head that is the identity: the rows' own 8-bit values, times their scale in fp32, rounded to the type."""
    torch = _torch()
    h = 336
    q = torch.eye(h, device="cuda").to(torch.float8_e4m3fn)
    s = torch.ones(3, 3, device="cuda")
    rng = np.random.default_rng(T)
    xb = to_bits(rng.normal(0, 1, (T, h)) * np.exp2(rng.integers(-6, 6, (T, h))), dtype)
    xb[0, :128] = 0
    x_q, x_s = O.fp8_blocks(O.widen(xb, dtype).astype(np.float32), 1)
    want = to_bits((x_q * np.repeat(x_s.astype(np.float64), 128, 1)[:, :h]).astype(np.float32), out)
    got = _lp().lp_lm_head_fp8_logits(to_dev_bits(xb, dtype), q, s, out_dtype=getattr(torch, OUT[out]))
    assert np.array_equal(host(got.double()), O.widen(want, out))


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,h", [(8, 4096), (16, 8192), (17, 4096), (32, 8192), (64, 4096), (128, 4096), (300, 4096), (300, 1280),
                                 (20, 8448), (5, 8448)])
def test_sums_that_cancel(out, T, h):
    """Each product comes a second time with the other sign, in another place: the logits are 0, and what comes out is error.
    Every block holds one x of 448 against a weight of 0, so that all have one scale and x is its own 8-bit value."""
    torch = _torch()
    V, n = 300, h // 2
    rng = np.random.default_rng(h + T)
    e4 = lambda a: torch.from_numpy(a.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()  # noqa: E731
    x, w = e4(np.clip(rng.normal(0, 60, (T, n)), -440, 440)), e4(np.clip(rng.normal(0, 110, (V, n)), -440, 440))
    x[:, ::128], w[:, ::128] = 448, 0
    at = np.concatenate([np.arange(b, b + 128) for b in rng.permutation(n // 128) * 128])
    at = at.reshape(-1, 128)
    at[:, 1:] = rng.permutation(at[:, 1:].reshape(-1)).reshape(at.shape[0], 127)  # any product anywhere but at the 448s
    at = at.reshape(-1)
    x, w = np.concatenate([x, x[:, at]], 1), np.concatenate([w, -w[:, at]], 1)
    assert not (x @ w.T).any()
    s = np.full((-(-V // 128), h // 128), 2.0 ** -12, dtype=np.float32)
    q = torch.from_numpy(w.astype(np.float32)).to(torch.float8_e4m3fn).cuda()
    got = _lp().lp_lm_head_fp8_logits(to_dev_bits(to_bits(x, "bf16"), "bf16"), q, torch.from_numpy(s).cuda(),
                                      out_dtype=getattr(torch, OUT[out]))
    rms = lambda a: float(np.sqrt(np.mean(np.square(a))))  # noqa: E731
    term = rms((x[:, :n] @ w[:, :n].T)) * np.sqrt(2) * float(s[0, 0])  # of a logit whose products were independent
    # fp32 sums: the i-th of a block's 128 is off by at most 2^-23 of about r sqrt(i), the j-th block's by that of r sqrt(128 j),
    # either way: 2^-23 r sqrt(h (64 + h / 256)) in all, of r sqrt(h)
    bound = 2.0 ** -23 * np.sqrt(64 + h / 256) * term
    if out != "fp32" and not (T <= 16 and h <= 8192):
        bound += 2.0 ** -13 * np.sqrt(8 / 3) * term
    got = host(got.double())
    assert rms(got) <= bound * (1 + EPS[out])
    print(f"rms of the error {rms(got) / term:.2e} of the logits' rms")
