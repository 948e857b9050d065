"""A NaN makes its row NaN, wherever it stands in the logits, in every call that
reduces rows."""
import numpy as np
import pytest

from tests.helpers import host, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V", [(12, 1031), (12, 5003), (12, 40009)])
def test_a_nan_shows(T, V):
    """Wherever it stands; its row only."""
    import entropy_chunked_row_amd as lp
    rng = np.random.default_rng(V + 2)
    x = rng.normal(0, 3, (T, V)).astype(np.float32)
    bad = np.arange(1, T, 2)
    x[bad, (bad * 211) % V] = np.nan
    y = np.full(T, 3, dtype=np.int64)
    y[bad] = (bad * 211 + 1) % V
    xd, yd = to_dev(x), to_dev(y)
    clean = to_dev(rng.normal(0, 3, (T, V)).astype(np.float32))
    a, H = lp.lp_logprobs_entropy(xd, yd)
    k, _ = lp.lp_logprobs_entropy_k(xd, yd.view(T, 1))
    for t in (a, H, k[:, 0], lp.lp_kl_full_vocab(xd, clean)[0], lp.lp_kl_full_vocab(clean, xd)[0]):
        t = host(t)
        assert np.isnan(t[bad]).all() and np.isfinite(np.delete(t, bad)).all()


@pytest.mark.parametrize("T,h,V", [(40, 256, 1024), (40, 72, 300), (300, 128, 5000)])
def test_a_nan_row_of_the_head_shows(T, h, V):
    """One vocabulary row of NaN makes one logit of every row NaN."""
    import torch

    import entropy_chunked_row_amd as lp
    hid, W = torch.randn(T, h, device="cuda").bfloat16(), (torch.randn(V, h, device="cuda") * 0.1).bfloat16()
    y = torch.zeros(T, dtype=torch.int64, device="cuda")
    good = lp.lp_lm_head_logprobs_entropy(hid, W, y, None, 1.0, 64)
    assert all(bool(torch.isfinite(t).all()) for t in good)
    for row in (V - 1, V // 2, 130):
        Wn = W.clone()
        Wn[row] = float("nan")
        for t in lp.lp_lm_head_logprobs_entropy(hid, Wn, y, None, 1.0, 64):
            assert bool(torch.isnan(t).all())
        assert bool(torch.isnan(lp.lp_lm_head_kl(hid, Wn, hid, W, None, None, None, 64)[0]).all())
        assert bool(torch.isnan(lp.lp_lm_head_kl(hid, W, hid, Wn, None, None, None, 64)[0]).all())
