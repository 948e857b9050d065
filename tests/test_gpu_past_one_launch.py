"""Calls of more rows or positions than one launch takes, and vocabularies at the
library's limit, against torch or against the same rows on their own."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.helpers import host, to_dev, to_dev_bits
from tests.rules_cases import to_bits

pytestmark = pytest.mark.gpu


def test_rules_of_many_rows():
    """More than 2^22 rows of three columns; each row's history is one token."""
    import torch

    import entropy_chunked_row_amd as lp
    T, V = (1 << 22) + 70001, 3
    x = torch.randn(T, V, device="cuda")
    tok = (torch.arange(T, device="cuda") % 5 - 1).int().view(T, 1)  # two of five ids lie outside
    one, pen = torch.ones(T, dtype=torch.int32, device="cuda"), torch.full((T,), 0.5, device="cuda")
    rules = lp.LogitRules(tokens=tok, hist_len=one, presence=pen)
    want = x.clone()
    ok = (tok >= 0) & (tok < V)
    want.scatter_add_(1, tok.clamp(0, V - 1).long(), torch.where(ok, -0.5, 0.0))
    assert torch.equal(lp.lp_process_logits(x, rules), want)
    y = torch.randint(0, V, (T,), device="cuda")
    a, H, lse = lp.lp_processed_logprobs_entropy(x, rules, y)
    logp = torch.log_softmax(want.double(), 1)
    assert (a.double() - logp.gather(1, y[:, None])[:, 0]).abs().max() <= 1e-5
    assert (H.double() + (logp.exp() * logp).sum(1)).abs().max() <= 1e-5
    d = lp.lp_processed_logprobs_entropy_backward(x, rules, y, None, 1.0, lse, H, pen)
    ref = -0.5 * logp.exp()
    ref.scatter_add_(1, y[:, None], torch.full((T, 1), 0.5, dtype=torch.float64, device="cuda"))
    assert (d.double() - ref).abs().max() <= 2e-5


def test_a_vocabulary_at_the_limit():
    import torch

    import entropy_chunked_row_amd as lp
    V = 1 << 30
    x = torch.zeros(1, V, dtype=torch.bfloat16, device="cuda")
    x[0, V - 3] = 30.0
    tok = torch.tensor([[V - 3, V - 3, 5, 163840]], dtype=torch.int32, device="cuda")
    half = torch.full((1,), 0.5, device="cuda")
    rules = lp.LogitRules(tokens=tok, hist_len=torch.full((1,), 4, dtype=torch.int32, device="cuda"), presence=half,
                          frequency=half)
    y = torch.tensor([V - 3], device="cuda")
    a, H, lse = (float(t) for t in lp.lp_processed_logprobs_entropy(x, rules, y))
    e = np.exp(28.5)  # 30 - 2 * 0.5 - 0.5
    s = e + (V - 3) + 2 * np.exp(-1.0)
    assert abs(lse - np.log(s)) <= 1e-5 and abs(a - (28.5 - np.log(s))) <= 1e-5
    assert abs(H - (np.log(s) - (28.5 * e - 2 * np.exp(-1.0)) / s)) <= 1e-5
    out = lp.lp_process_logits(x, rules)
    assert out[0, [V - 3, 5, 163840, 6, V - 1]].tolist() == [28.5, -1.0, -1.0, 0.0, 0.0]
    out[0, [V - 3, 5, 163840]] = 0
    assert not out.any()


def test_embedding_gradient_of_many_positions():
    """More than 2^23 spans of 16 sorted positions; whole numbers, so sums are exact."""
    import torch

    import entropy_chunked_row_amd as lp
    N, V = (1 << 27) + 100003, 1000
    tok = torch.randint(-1, V + 1, (N,), device="cuda")
    g = (torch.arange(N, device="cuda") % 3 - 1).to(torch.bfloat16).view(N, 1)
    got = lp.lp_embedding_backward(g, tok, V)
    ok = (tok >= 0) & (tok < V)
    want = torch.bincount(torch.where(ok, tok, V), weights=g[:, 0].double(), minlength=V + 1)[:V]
    assert torch.equal(got[:, 0].double(), want)


def test_embedding_gradient_of_a_wide_vocabulary():
    import torch

    import entropy_chunked_row_amd as lp
    V, N = 1 << 30, 5000
    tok = torch.randint(0, V, (N,), device="cuda")
    tok[:3] = torch.tensor([V - 1, 0, V], device="cuda")
    tok[3000:] = tok[:2000]
    g = torch.ones(N, 1, device="cuda")
    got = lp.lp_embedding_backward(g, tok, V)
    ids, n = tok[tok < V].unique(return_counts=True)
    assert torch.equal(got[ids, 0], n.float()) and int(got.sum(dtype=torch.float64)) == int(n.sum())


def test_head_of_many_rows():
    """More than 65535 blocks of 64 rows."""
    import torch

    import entropy_chunked_row_amd as lp
    T, h, V = 65535 * 64 + 77, 32, 17
    rng = np.random.default_rng(1)
    q = rng.integers(0, 16, (V, h))
    packed = to_dev((q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8))
    scales = torch.full((V, 1), 0.5, dtype=torch.bfloat16, device="cuda")
    x = (torch.arange(T * h, device="cuda") % 7 - 3).to(torch.bfloat16).view(T, h)
    got = lp.lp_lm_head_w4_logits(x, packed, scales, 32, out_dtype=torch.float32)
    want = x.float() @ to_dev((q - 8).astype(np.float32)).t() * 0.5  # whole numbers: exact
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,tiny", [("bf16", 2.0 ** -133), ("fp16", 2.0 ** -24)])
@pytest.mark.parametrize("T", [1, 40])
def test_subnormal_hidden_states(dtype, tiny, T):
    """The smallest steps of the type count: 5 times the smallest number, times
    scales that bring the products back."""
    import torch

    import entropy_chunked_row_amd as lp
    h, V = 64, 33
    rng = np.random.default_rng(2)
    q = rng.integers(0, 16, (V, h))
    s = np.full((V, 2), 2.0 ** 20)
    x = rng.integers(-5, 6, (T, h)) * tiny
    xb = to_bits(x, dtype)
    assert np.array_equal(O.widen(xb, dtype), x)
    got = lp.lp_lm_head_w4_logits(to_dev_bits(xb, dtype), to_dev((q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)),
                                  to_dev_bits(to_bits(s, "bf16"), "bf16"), 32, out_dtype=torch.float32)
    assert np.array_equal(host(got).astype(np.float64), O.w4_logits(x, q, s, 32))
