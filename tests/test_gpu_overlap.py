"""Operands and outputs that lie beside each other in the rows of one buffer
share no bytes, and are taken."""
import pytest

from tests.helpers import to_dev
from tests.rules_cases import DTYPES, Rules

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gap", [0, 1, 8])
def test_rules_beside_their_logits(dtype, gap):
    import torch

    import entropy_chunked_row_amd as lp
    V, T = 1031, 9
    c = Rules(T, V, dtype, seed=11, empty_row=False)
    x, rules = c.device()
    want = lp.lp_process_logits(x, rules)
    y, g = to_dev(c.targets), torch.linspace(-1, 1, T, device="cuda")
    a = lp.lp_processed_logprobs_entropy(x, rules, y, None, 0.7)
    grad = lp.lp_processed_logprobs_entropy_backward(x, rules, y, None, 0.7, a[2], a[1], g, g)
    for first in (True, False):
        buf = torch.full((T, 2 * V + gap), 5.0, dtype=x.dtype, device="cuda")
        left, right = buf[:, :V], buf[:, V + gap:]
        src, dst = (left, right) if first else (right, left)
        src.copy_(x)
        lp.lp_process_logits(src, rules, out=dst)
        assert torch.equal(dst.float(), want.float()) and torch.equal(src.float(), x.float())
        lp.lp_processed_logprobs_entropy_backward(src, rules, y, None, 0.7, a[2], a[1], g, g, grad_logits=dst)
        assert torch.equal(dst, grad) and torch.equal(src.float(), x.float())
        assert bool((buf[:, V:V + gap] == 5).all())
        with pytest.raises(lp.LPError, match="overlaps"):
            lp.lp_process_logits(buf[:, :V], rules, out=buf[:, V - 1:2 * V - 1])


def test_embedding_and_head_beside_their_operands():
    import torch

    import entropy_chunked_row_amd as lp
    buf = torch.randn(300, 200, device="cuda").bfloat16()
    tok = torch.randint(0, 300, (300,), device="cuda")
    want = lp.lp_embedding(buf[:, :96].contiguous(), tok, 2.0)
    lp.lp_embedding(buf[:, :96], tok, 2.0, out=buf[:, 97:193])
    assert torch.equal(buf[:, 97:193], want)
    with pytest.raises(lp.LPError, match="overlaps"):
        lp.lp_embedding(buf[:, :96], tok, 2.0, out=buf[:, 95:191])
    g = torch.randn(50, 64, device="cuda")
    with pytest.raises(lp.LPError, match="overlaps"):
        lp.lp_embedding_backward(g, tok[:50] % 10, 10, 1.0, grad_weight=g[5:15])
    x = torch.randn(4, 64, device="cuda").half()
    p, s = lp.lp_lm_head_w4_quantize(torch.randn(64, 64, device="cuda"), 32)
    with pytest.raises(lp.LPError, match="overlaps"):
        lp.lp_lm_head_w4_logits(x, p, s, 32, out=x)
    with pytest.raises(lp.LPError, match="overlap"):
        lp.lp_lm_head_w4_quantize(x, 32, packed=x.view(torch.uint8)[:, :32])
