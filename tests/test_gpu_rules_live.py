"""A LogitRules whose tensors were resized, replaced or filled anew after it
was made gives what one made of them now would give."""
import numpy as np
import pytest

from tests.helpers import to_dev
from tests.rules_cases import Rules

pytestmark = pytest.mark.gpu


def test_tensors_as_they_are_at_the_call():
    import torch

    import entropy_chunked_row_amd as lp
    V = 3001
    first, second = Rules(5, V, "fp32", seed=1, empty_row=False), Rules(70, V, "fp32", seed=2, L=90, empty_row=False)
    x, rules = first.device()
    kept = dict(rules._whole + rules._per_row)
    before = lp.lp_process_logits(x, rules)
    x2, fresh = second.device()
    want = lp.lp_process_logits(x2, fresh)
    # grown in place, then filled
    for name, t in dict(fresh._whole + fresh._per_row).items():
        kept[name].resize_(t.shape).copy_(t)
    assert torch.equal(lp.lp_process_logits(x2, rules), want)
    y = to_dev(second.targets)
    for a, b in zip(lp.lp_processed_logprobs_entropy(x2, rules, y, None, 0.7),
                    lp.lp_processed_logprobs_entropy(x2, fresh, y, None, 0.7)):
        assert torch.equal(a, b)
    # pointed at other storage
    _, again = first.device()
    for name, t in dict(again._whole + again._per_row).items():
        kept[name].data = t
    assert torch.equal(lp.lp_process_logits(x, rules), before)
    with pytest.raises(ValueError):
        lp.lp_process_logits(x2, rules)
    # new values in place
    kept["hist_len"].zero_()
    kept["bias_values"].zero_()
    kept["allowed"].fill_(-1)
    assert torch.equal(lp.lp_process_logits(x, rules), x) and np.isfinite(float(x.sum()))
