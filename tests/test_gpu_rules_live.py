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


def test_one_set_of_rules_in_two_threads():
    """Calls made at once from two threads, each on a stream of its own, share the rules and nothing else."""
    import threading

    import torch

    import entropy_chunked_row_amd as lp
    c = Rules(40, 5003, "bf16", seed=9, L=200, empty_row=False)
    x, rules = c.device()
    xs = [x, x.flip(1).contiguous()]
    y = to_dev(c.targets)
    want = [lp.lp_process_logits(t, rules) for t in xs], [lp.lp_processed_logprobs_entropy(t, rules, y) for t in xs]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        stream = torch.cuda.Stream()
        for _ in range(30):
            z = lp.lp_process_logits(xs[k], rules, stream=stream)
            s = lp.lp_processed_logprobs_entropy(xs[k], rules, y, stream=stream)
            stream.synchronize()
            if not torch.equal(z, want[0][k]) or not all(torch.equal(a, b) for a, b in zip(s, want[1][k])):
                wrong.append(k)
                return

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong
