"""CPU checks of choosing from rows, distillation and beams: worked values of the
oracle, its gradient against differences, and every refusal."""
import math

import numpy as np
import pytest
import torch

import entropy_chunked_row_amd as lp
from oracle import lp_oracle as O

FAKE = 0x10000  # never dereferenced


def test_oracle_top_of_a_row():
    z = np.array([[1.0, 3.0, 3.0, -np.inf, 0.0, 2.0], [5.0] * 6])
    ids, lpk, rest, lse = O.top_logits(z, 3, None, 1.0)
    assert ids.tolist() == [[1, 2, 5], [0, 1, 2]]
    s = math.exp(1) + 2 * math.exp(3) + 1 + math.exp(2)
    assert np.allclose(lpk[0], [3 - math.log(s), 3 - math.log(s), 2 - math.log(s)], atol=1e-14)
    assert np.isclose(rest[0], math.log((math.exp(1) + 1) / s)) and np.isclose(rest[1], math.log(0.5))
    ids, lpk, rest, _ = O.top_logits(z[:1, 2:4], 2, None, 1.0)
    assert ids.tolist() == [[0, -1]] and lpk[0].tolist() == [0.0, -np.inf] and rest[0] == -np.inf


def test_oracle_distillation_against_full_kl():
    """A list of the whole vocabulary is the exact KL; a shorter one merges the rest into one outcome and can only lose."""
    rng = np.random.default_rng(3)
    u, v = rng.normal(0, 2, (4, 9)), rng.normal(0, 2, (4, 9))
    logp = O.log_softmax(v)
    ids = np.tile(np.arange(9), (4, 1))
    full = O.distill_top(u, ids, logp, None, None, 1.0)[0]
    assert np.allclose(full, O.kl_full_vocab(u, v), atol=1e-12)
    ids, lpk, rest, _ = O.top_logits(v, 4, None, 1.0)
    part = O.distill_top(u, ids, lpk, rest, None, 1.0)[0]
    p = np.exp(lpk)
    q = np.exp(np.take_along_axis(O.log_softmax(u), ids, 1))
    want = (p * np.log(p / q)).sum(1) + (1 - p.sum(1)) * np.log((1 - p.sum(1)) / (1 - q.sum(1)))
    assert np.allclose(part, want, atol=1e-12) and np.all(part <= full + 1e-12) and np.all(part >= 0)
    assert np.allclose(O.distill_top(v, ids, lpk, rest, None, 1.0)[0], 0, atol=1e-12)


@pytest.mark.parametrize("tau", [1.0, 0.7, 1.6])
@pytest.mark.parametrize("with_rest", [True, False])
def test_oracle_distillation_gradient_against_differences(tau, with_rest):
    rng = np.random.default_rng(5)
    z = rng.normal(0, 1.5, (3, 8))
    ids = np.array([[1, 4, 1, -1], [0, 7, 2, 3], [5, 8, 6, 6]])  # an id twice, ids outside
    lpk, rest = np.log(rng.uniform(0.05, 0.3, (3, 4))), np.log(rng.uniform(0.05, 0.3, 3))
    lpk[1, 2] = -np.inf
    rest = rest if with_rest else None
    g, mask = rng.normal(0, 1, 3), np.array([1, 1, 1])
    d = O.distill_top_backward(z, ids, lpk, rest, mask, tau, g)
    f = lambda x: (O.distill_top(x, ids, lpk, rest, mask, tau)[0] * g).sum()  # noqa: E731
    for t in range(3):
        for j in range(8):
            e = np.zeros_like(z)
            e[t, j] = 1e-5
            assert abs((f(z + e) - f(z - e)) / 2e-5 - d[t, j]) <= 1e-8
    # a shift of a row changes nothing
    assert np.allclose(d.sum(1), 0, atol=1e-12)


def test_oracle_beams():
    z = np.log(np.array([[0.5, 0.3, 0.2], [0.6, 0.4, 1e-300]]))
    s, p, y = O.beam_select(z, np.array([[-1.0, -1.1]]), 4, None, 0, 1.0)
    assert p.tolist() == [[1, 0, 1, 0]] and y.tolist() == [[0, 0, 1, 1]]
    assert np.allclose(s[0], [-1.1 + math.log(0.6), -1 + math.log(0.5), -1.1 + math.log(0.4), -1 + math.log(0.3)])
    s, p, y = O.beam_select(z, np.array([[-0.5, -9.0]]), 3, np.array([[1, 0]]), 2, 1.0)
    assert p.tolist() == [[0, 1, 1]] and y.tolist() == [[2, 0, 1]] and s[0, 0] == -0.5
    s, p, y = O.beam_select(z, np.array([[-np.inf, np.nan]]), 2, None, 0, 1.0)
    assert p.tolist() == [[-1, -1]] and y.tolist() == [[-1, -1]] and np.all(s == -np.inf)
    out = O.beam_reorder(np.arange(8).reshape(4, 2), np.array([[1, 1, 0], [0, -1, 2]]), 0)
    assert out.tolist() == [[2, 3], [2, 3], [0, 1], [4, 5], [0, 0], [0, 0]]


# --- refusals ------------------------------------------------------------

def test_binding_refusals_of_top():
    z = torch.zeros(3, 10)
    for bad in (z[0], z.t(), z[:, ::2]):
        with pytest.raises(ValueError, match="2-D"):
            lp.lp_top_logits(bad, 2)
    with pytest.raises(TypeError):
        lp.lp_top_logits(z.double(), 2)
    with pytest.raises(ValueError, match="mask"):
        lp.lp_top_logits(z, 2, torch.ones(4, dtype=torch.uint8))
    with pytest.raises(TypeError, match="mask"):
        lp.lp_top_logits(z, 2, torch.ones(3))
    with pytest.raises(ValueError, match="device"):
        lp.lp_top_logits(z, 2)


def test_binding_refusals_of_distillation():
    z, ids, p = torch.zeros(3, 10), torch.zeros(3, 4, dtype=torch.int64), torch.zeros(3, 4)
    v = torch.zeros(3)
    cases = [(dict(teacher_ids=ids[0]), "teacher_ids"), (dict(teacher_ids=ids[:2]), "teacher_ids"),
             (dict(teacher_logprob=p[:, :3].contiguous()), "teacher_logprob"), (dict(teacher_logprob=p.view(4, 3)), "teacher_logprob"),
             (dict(teacher_rest=torch.zeros(4)), "teacher_rest"), (dict(mask=torch.ones(2, dtype=torch.uint8)), "mask"),
             (dict(teacher_ids=ids.t().contiguous().t()), "contiguous"), (dict(), "device")]
    for over, match in cases:
        kw = dict(teacher_ids=ids, teacher_logprob=p, teacher_rest=None, mask=None)
        kw.update(over)
        with pytest.raises(ValueError, match=match):
            lp.lp_distill_top(z, **kw)
        with pytest.raises(ValueError, match=match):
            lp.lp_distill_top_backward(z, temperature=1.0, lse=v, lse_rest=v, grad_loss=v, **kw)
    for bad in (dict(teacher_ids=ids.int()), dict(teacher_logprob=p.double()), dict(teacher_rest=v.double())):
        kw = dict(teacher_ids=ids, teacher_logprob=p, teacher_rest=None)
        kw.update(bad)
        with pytest.raises(TypeError):
            lp.lp_distill_top(z, **kw)
    good = dict(teacher_rest=None, mask=None, temperature=1.0, lse=v, lse_rest=v, grad_loss=v)
    for name in ("lse", "lse_rest", "grad_loss"):
        with pytest.raises(ValueError, match=name):
            lp.lp_distill_top_backward(z, ids, p, **{**good, name: torch.zeros(2)})
    with pytest.raises(ValueError, match="grad_logits"):
        lp.lp_distill_top_backward(z, ids, p, **good, grad_logits=torch.zeros(3, 11))
    with pytest.raises(ValueError, match="grad_logits"):
        lp.lp_distill_top_backward(z, ids, p, **good, grad_logits=torch.zeros(3, 10).half())


def test_binding_refusals_of_beams():
    z, s = torch.zeros(6, 10), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="beam_scores"):
        lp.lp_beam_select(z, torch.zeros(6))
    with pytest.raises(ValueError, match="beam_scores"):
        lp.lp_beam_select(z, torch.zeros(2, 4))
    with pytest.raises(TypeError, match="beam_scores"):
        lp.lp_beam_select(z, s.double())
    with pytest.raises(ValueError, match="finished"):
        lp.lp_beam_select(z, s, 3, torch.zeros(2, 2, dtype=torch.bool))
    with pytest.raises(ValueError, match="device"):
        lp.lp_beam_select(z, s)
    x, p = torch.zeros(5, 6, 4, 7), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="parents"):
        lp.lp_beam_reorder(x, p[0], dim=1)
    with pytest.raises(TypeError, match="parents"):
        lp.lp_beam_reorder(x, p.long(), dim=1)
    with pytest.raises(ValueError, match="no beams"):
        lp.lp_beam_reorder(x, p, dim=0)
    with pytest.raises(ValueError, match="dim"):
        lp.lp_beam_reorder(x, p, dim=4)
    with pytest.raises(ValueError, match="out must"):
        lp.lp_beam_reorder(x, p, dim=1, out=torch.zeros(5, 6, 4, 8))
    with pytest.raises(ValueError, match="out must"):
        lp.lp_beam_reorder(x, p, dim=1, out=x.int())
    with pytest.raises(ValueError, match="one step"):
        lp.lp_beam_reorder(torch.zeros(2, 6, 4, 5, 7)[:, :, ::2, ::2, :3], p, dim=1)
    with pytest.raises(ValueError, match="one step"):
        lp.lp_beam_reorder(torch.zeros(4, 5, 6, 2)[::2, ::2], p, dim=2)
    with pytest.raises(ValueError, match="device"):
        lp.lp_beam_reorder(x, p, dim=1)


def _top(L, **over):
    d = dict(x=FAKE, dtype=0, T=3, V=10, ld=10, K=4, mask=None, tau=1.0, ids=0x20000, p=0x30000, rest=0x40000, lse=0x50000,
             ws=0x60000, n=1 << 20)
    d.update(over)
    return L.lp_top_logits(d["x"], d["dtype"], d["T"], d["V"], d["ld"], d["K"], d["mask"], d["tau"], d["ids"], d["p"], d["rest"],
                           d["lse"], d["ws"], d["n"], None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=7), 1), (dict(T=-1), 1), (dict(V=0), 1), (dict(V=2**31), 1), (dict(ld=9), 1), (dict(K=0), 1), (dict(K=11), 1),
    (dict(K=257, V=1000, ld=1000), 1), (dict(tau=float("nan")), 1), (dict(tau=float("inf")), 1), (dict(x=None), 1),
    (dict(x=FAKE + 1), 1), (dict(ids=None), 1), (dict(p=None), 1), (dict(ids=0x20004), 1), (dict(p=0x30002), 1),
    (dict(rest=0x40001), 1), (dict(lse=0x50001), 1), (dict(ws=None), 3), (dict(n=255), 3), (dict(ws=0x60080), 1),
    (dict(T=2**41), 2), (dict(ld=2**40), 2), (dict(ids=FAKE), 1), (dict(p=0x20010), 1), (dict(ws=0x20000), 1),
    (dict(rest=0x50000), 1), (dict(mask=0x40000), 1), (dict(T=0, x=None, ids=None, p=None, ws=None), 0)])
def test_c_refusals_of_top(lib_handle, over, code):
    assert _top(lib_handle, **over) == code
    assert code == 0 or lib_handle.lp_last_error() != b""


@pytest.mark.parametrize("over,code", [
    (dict(dtype=7), 1), (dict(T=-1), 1), (dict(V=0), 1), (dict(ld=9), 1), (dict(K=0), 1), (dict(K=257), 1),
    (dict(tau=float("nan")), 1), (dict(x=None), 1), (dict(x=FAKE + 1), 1), (dict(ids=None), 1), (dict(p=None), 1),
    (dict(ids=0x20004), 1), (dict(p=0x30002), 1), (dict(rest=0x40001), 1), (dict(T=2**41), 2),
    (dict(T=0, x=None, ids=None, p=None, out=None, lse=None, lser=None, g=None, ws=None), 0),
    (dict(out=None), 1), (dict(out=0x50001), 1), (dict(lse=0x70001), 1), (dict(lser=0x80001), 1), (dict(out=FAKE + 4), 1),
    (dict(out=0x20008), 1), (dict(out=0x30008), 1), (dict(out=0x40004), 1)])
def test_c_refusals_of_distillation(lib_handle, over, code):
    d = dict(x=FAKE, dtype=0, T=3, V=10, ld=10, K=4, ids=0x20000, p=0x30000, rest=0x40000, mask=None, tau=1.0, out=0x50000,
             lse=0x70000, lser=0x80000, g=0x90000, ws=0x60000)
    d.update(over)
    lead = (d["x"], d["dtype"], d["T"], d["V"], d["ld"], d["K"], d["ids"], d["p"], d["rest"], d["mask"], d["tau"])
    assert lib_handle.lp_distill_top(*lead, d["out"], d["lse"], d["lser"], d["ws"], 1 << 20, None) == code
    assert lib_handle.lp_distill_top_backward(*lead, d["lse"], d["lser"], d["g"], d["out"], 10, None) == code


def test_c_refusals_of_distillation_apart(lib_handle):
    lead = (FAKE, 0, 3, 10, 10, 4, 0x20000, 0x30000, 0x40000, None, 1.0)
    f, b = lib_handle.lp_distill_top, lib_handle.lp_distill_top_backward
    assert f(*lead, 0x50000, None, None, None, 1 << 20, None) == 3
    assert f(*lead, 0x50000, None, None, 0x60000, 255, None) == 3
    assert f(*lead, 0x50000, None, None, 0x60010, 1 << 20, None) == 1
    assert f(*lead, 0x50000, 0x50004, None, 0x60000, 1 << 20, None) == 1
    assert b(*lead, 0x70000, 0x80000, 0x90000, 0x50000, 9, None) == 1
    assert b(*lead, 0x70000, 0x80000, 0x90000, 0x50000, 2**40, None) == 2
    for k in range(3):
        v = [0x70000, 0x80000, 0x90000]
        v[k] = None
        assert b(*lead, *v, 0x50000, 10, None) == 1
        v[k] = 0x50004
        assert b(*lead, *v, 0x50000, 10, None) == 1


@pytest.mark.parametrize("over,code", [
    (dict(dtype=5), 1), (dict(B=-1), 1), (dict(W=0), 1), (dict(W=65), 1), (dict(N=0), 1), (dict(N=257), 1),
    (dict(W=64, N=65), 1), (dict(V=0), 1), (dict(ld=9), 1), (dict(end=-1), 1), (dict(end=10), 1), (dict(tau=float("nan")), 1),
    (dict(x=None), 1), (dict(s=None), 1), (dict(s=0x20001), 1), (dict(out=None), 1), (dict(par=None), 1), (dict(tok=None), 1),
    (dict(tok=0x50004), 1), (dict(ws=None), 3), (dict(n=255), 3), (dict(ws=0x60010), 1), (dict(out=0x20000), 1),
    (dict(par=0x50000), 1), (dict(ws=0x30000), 1), (dict(fin=0x30000), 1), (dict(B=2**35), 1),
    (dict(B=0, x=None, s=None, out=None, par=None, tok=None, ws=None), 0)])
def test_c_refusals_of_beams(lib_handle, over, code):
    d = dict(x=FAKE, dtype=0, B=2, W=3, V=10, ld=10, s=0x20000, fin=None, N=4, end=0, tau=1.0, out=0x30000, par=0x40000,
             tok=0x50000, ws=0x60000, n=1 << 20)
    d.update(over)
    assert lib_handle.lp_beam_select(d["x"], d["dtype"], d["B"], d["W"], d["V"], d["ld"], d["s"], d["fin"], d["N"], d["end"],
                                     d["tau"], d["out"], d["par"], d["tok"], d["ws"], d["n"], None) == code


@pytest.mark.parametrize("over,code", [
    (dict(W=0), 1), (dict(W=257), 1), (dict(N=0), 1), (dict(N=257), 1), (dict(B=-1), 1), (dict(outer=-1), 1), (dict(mid=-1), 1),
    (dict(width=-1), 1), (dict(so=-8), 1), (dict(sr=2**41), 1), (dict(src=None), 1), (dict(dst=None), 1), (dict(par=None), 1),
    (dict(par=0x90002), 1), (dict(dm=7), 1), (dict(dr=15), 1), (dict(do=95), 1), (dict(dst=FAKE + 100), 1), (dict(par=0x20000), 1),
    (dict(B=2**20, mid=2**11), 2), (dict(width=2**36, dm=2**36, dr=2**38, outer=1, dst=2**45), 2),
    (dict(B=0, src=None), 0), (dict(width=0, src=None), 0), (dict(outer=0, dst=None), 0)])
def test_c_refusals_of_reordering(lib_handle, over, code):
    d = dict(src=FAKE, so=96, sr=16, sm=8, outer=3, mid=2, width=8, par=0x90000, B=2, W=3, N=3, dst=0x20000, do=96, dr=16, dm=8)
    d.update(over)
    assert lib_handle.lp_beam_reorder(d["src"], d["so"], d["sr"], d["sm"], d["outer"], d["mid"], d["width"], d["par"], d["B"],
                                      d["W"], d["N"], d["dst"], d["do"], d["dr"], d["dm"], None) == code


def test_workspace_sizes(lib_handle):
    L = lib_handle
    assert L.lp_top_workspace_bytes(0, 8192, 151936, 64) == 256  # a row a workgroup
    assert L.lp_top_workspace_bytes(0, 1, 151936, 64) % 256 == 0 and L.lp_top_workspace_bytes(0, 1, 151936, 64) > 256
    for bad in ((7, 1, 10, 1), (0, -1, 10, 1), (0, 1, 0, 1), (0, 1, 10, 11), (0, 1, 1000, 257), (0, 2**41, 10, 1)):
        assert L.lp_top_workspace_bytes(*bad) == 0
    assert L.lp_distill_top_workspace_bytes(0, 8192, 151936) == 256 and L.lp_distill_top_workspace_bytes(0, 1, 151936) > 256
    for bad in ((7, 1, 10), (0, -1, 10), (0, 1, 0), (0, 2**41, 10)):
        assert L.lp_distill_top_workspace_bytes(*bad) == 0
    assert L.lp_beam_workspace_bytes(0, 64, 8, 129280, 16) > 0
    for bad in ((7, 1, 1, 10, 1), (0, -1, 1, 10, 1), (0, 1, 65, 10, 1), (0, 1, 64, 10, 65), (0, 1, 1, 0, 1)):
        assert L.lp_beam_workspace_bytes(*bad) == 0


def test_no_streamed_slice_is_shorter_than_a_step(lib_handle):
    """Slices of a row are kept whole (at most 4 vectors a thread: 256 threads up to K = 64, else 512), or all of them
    hold a step of the stream, as many columns.  Seen through the workspace, which has 8 K + 8 bytes a slice."""
    rng = np.random.default_rng(0)
    cases = [(2, 80, 60740, 22), (0, 68, 135830, 43), (2, 35, 159221, 225), (0, 1, 151936, 20), (1, 1, 8193, 5)]
    for _ in range(3000):
        V = int(2 ** rng.uniform(10, 18))
        cases.append((int(rng.integers(0, 3)), int(2 ** rng.uniform(0, 10)), V, int(rng.integers(1, min(256, V) + 1))))
    for dtype, T, V, K in cases:
        size = lib_handle.lp_top_workspace_bytes(dtype, T, V, K)
        per = T * (8 * K + 8)
        counts = [n for n in range(2, 1025) if -(-n * per // 256) * 256 == size]
        if len(counts) != 1:
            continue  # one slice, or sizes that say nothing
        n = counts[0]
        kept = 4 * (512 if K > 64 else 256) * (4 if dtype == 2 else 8)
        slices = [s for s in range(64, V + 64, 64) if -(-V // s) == n] if T < 4 else [-(-(-(-V // n)) // 64) * 64]
        assert any(s <= kept or V - (n - 1) * s >= kept for s in slices), (dtype, T, V, K, n)
