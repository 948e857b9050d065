"""CPU checks of the embedding calls: the oracle against differences, and every
refusal of the binding and of the C entry points."""
import numpy as np
import pytest
import torch

import entropy_chunked_row_amd as lp
from oracle import lp_oracle as O

FAKE = 0x10000  # never dereferenced


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(2)
    W, tok, c = rng.normal(size=(5, 3)), np.array([1, 4, 1, -1, 5]), rng.normal(size=(5, 3))
    d = O.embedding_backward(c, tok, 5, 1.5)
    for v in range(5):
        for j in range(3):
            up, dn = W.copy(), W.copy()
            up[v, j] += 0.5
            dn[v, j] -= 0.5
            diff = ((O.embedding(up, tok, 1.5) - O.embedding(dn, tok, 1.5)) * c).sum()
            assert abs(diff - d[v, j]) < 1e-12


def test_binding_refusals():
    w, g, t = torch.zeros(10, 8), torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        lp.lp_embedding(w.double(), t)
    with pytest.raises(TypeError, match="int64"):
        lp.lp_embedding(w, t.int())
    with pytest.raises(ValueError, match="contiguous rows"):
        lp.lp_embedding(w.t(), t)
    with pytest.raises(ValueError, match="contiguous"):
        lp.lp_embedding(w, torch.zeros(8, dtype=torch.int64)[::2])
    with pytest.raises(ValueError, match="out must be"):
        lp.lp_embedding(w, t, out=torch.zeros(4, 7))
    with pytest.raises(ValueError, match="device"):
        lp.lp_embedding(w, t)
    with pytest.raises(ValueError, match="elements"):
        lp.lp_embedding_backward(g, t[:3], 10)
    with pytest.raises(ValueError, match="accumulate"):
        lp.lp_embedding_backward(g, t, 10, accumulate=True)
    with pytest.raises(ValueError, match="grad_weight"):
        lp.lp_embedding_backward(g, t, 10, grad_weight=torch.zeros(8, 10))
    with pytest.raises(TypeError, match="float32"):
        lp.lp_embedding_backward(g, t, 10, grad_weight=torch.zeros(10, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous"):
        lp.lp_embedding_backward(torch.zeros(2, 8, 2).transpose(1, 2), t, 10)
    with pytest.raises(ValueError, match="device"):
        lp.lp_embedding_backward(g, t, 10)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=5), 1), (dict(V=0), 1), (dict(V=2**31), 1), (dict(h=0), 1), (dict(N=-1), 1), (dict(ld=7), 1),
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(a=None), 1), (dict(tok=None), 1),
    (dict(out=None), 1), (dict(a=FAKE + 1), 1), (dict(tok=FAKE + 4), 1), (dict(out=FAKE + 1), 1), (dict(ld=2**60), 2)])
def test_c_refusals(lib_handle, over, code):
    d = dict(a=FAKE, dtype=0, V=10, h=8, ld=8, tok=FAKE, N=4, scale=1.0, out=FAKE)
    d.update(over)
    assert lib_handle.lp_embedding(d["a"], d["dtype"], d["V"], d["h"], d["ld"], d["tok"], d["N"], d["scale"], d["out"],
                                   max(d["ld"], 8), None) == code
    assert lib_handle.lp_embedding_backward(d["a"], d["dtype"], d["N"], d["h"], d["ld"], d["tok"], d["V"], d["scale"], 0,
                                            d["out"], FAKE, 1 << 40, None) == code
    assert lib_handle.lp_last_error() != b""


def test_c_workspace_and_empty(lib_handle):
    L = lib_handle
    f = L.lp_embedding_workspace_bytes
    assert f(-1, 8, 8) == 0 and f(4, 0, 8) == 0 and f(4, 8, 0) == 0 and f(2**31, 8, 8) == 0
    need = f(5000, 8, 10)
    assert need % 256 == 0 and need >= 4 * 5000 * 4
    call = lambda ws, n: L.lp_embedding_backward(FAKE, 0, 5000, 8, 8, FAKE, 10, 1.0, 0, FAKE, ws, n, None)  # noqa: E731
    assert call(FAKE, need - 1) == 3 and call(None, need) == 3 and call(FAKE + 64, need) == 1
    assert L.lp_embedding_backward(FAKE, 0, 2**31, 8, 8, FAKE, 10, 1.0, 0, FAKE, FAKE, 1 << 40, None) == 2
    assert L.lp_embedding(None, 0, 10, 8, 8, None, 0, 1.0, None, 8, None) == 0
    assert L.lp_embedding_backward(None, 0, 0, 8, 8, None, 10, 1.0, 1, FAKE, None, 0, None) == 0
    assert L.lp_embedding_backward(None, 0, 0, 8, 8, None, 10, 1.0, 0, None, None, 0, None) == 1
