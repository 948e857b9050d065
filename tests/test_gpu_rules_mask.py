"""Processed logits without an output of the caller's: rows of mask 0 are 0,
whatever the memory held before; also when captured and replayed."""
import pytest

from tests.helpers import host, to_dev
from tests.rules_cases import DTYPES, Rules

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V", [(9, 1031), (1, 9001), (300, 5003)])
def test_unscored_rows_are_zero(dtype, T, V):
    import torch

    import entropy_chunked_row_amd as lp
    c = Rules(T, V, dtype, seed=T)
    c.mask[0] = 0
    x, rules = c.device()
    m = to_dev(c.mask)
    want = lp.lp_process_logits(x, rules)
    on = torch.from_numpy(c.mask != 0).cuda()
    for _ in range(4):
        dirty = torch.full((T, V), float("nan"), dtype=x.dtype, device="cuda")
        del dirty  # its memory is the next allocation's
        got = lp.lp_process_logits(x, rules, m)
        assert not got[~on].any() and torch.equal(got[on].float(), want[on].float())
    assert lp.lp_process_logits(x, rules, torch.zeros_like(m)).any().item() is False


def test_captured():
    import torch

    import entropy_chunked_row_amd as lp
    c = Rules(20, 3001, "bf16", seed=3)
    x, rules = c.device()
    m = to_dev(c.mask)
    lp.lp_process_logits(x, rules, m)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lp.lp_process_logits(x, rules, m)
    for k in range(4):
        m.copy_(to_dev((c.mask + k) % 2))
        got.fill_(float("nan"))
        eager = lp.lp_process_logits(x, rules, m)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.float(), eager.float()) and not host(got.float())[host(m) == 0].any()
