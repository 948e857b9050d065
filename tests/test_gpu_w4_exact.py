"""The 4-bit head where nothing is rounded: whole numbers of x, power-of-two
scales, every sum below 2^24 steps.  fp32 logits are then equal to the last bit,
at real widths, and a single misplaced nibble shows."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.helpers import host, to_dev, to_dev_bits
from tests.rules_cases import to_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("h", [992, 5120, 7168, 8192])
def test_equal_to_the_bit(dtype, group, h):
    import torch

    import entropy_chunked_row_amd as lp
    rng = np.random.default_rng(h + group)
    V = 301
    q = rng.integers(0, 16, (V, h))
    # |x| (16 + q) <= 62 and the shift 24 |x| <= 48 in steps of 2^-3: 8192 * 110 * 2^3 < 2^24
    s = 2.0 ** rng.integers(-3, 1, (V, -(-h // group)))
    x = rng.integers(-2, 3, (70, h)).astype(np.float64)
    packed = to_dev((q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8))
    scales = to_dev_bits(to_bits(s, "bf16"), "bf16")
    hid = to_dev_bits(to_bits(x, dtype), dtype)
    want = O.w4_logits(x, q, s, group)
    for T in (1, 8, 16, 17, 40, 64, 70):
        got = lp.lp_lm_head_w4_logits(hid[:T], packed, scales, group, out_dtype=torch.float32)
        assert np.array_equal(host(got).astype(np.float64), want[:T]), T
