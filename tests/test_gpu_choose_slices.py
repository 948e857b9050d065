"""Rows that are cut into slices and joined: special values, ties, short last slices, graphs, streams and workspaces.  Each test
first makes sure, by the workspace that the call asks for (256 bytes where nothing is joined), that its rows are cut."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.choose_cases import SUM, close, dev_rows, grad_tol, lists, peaked, tol_log
from tests.helpers import host, to_dev, to_dev_bits
from tests.rules_cases import DTYPES, to_bits

pytestmark = pytest.mark.gpu
CODE = {"bf16": 0, "fp16": 1, "fp32": 2}


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def _torch():
    import torch
    return torch


def _cut(dtype, T, V, K):
    assert _lp().lp_top_workspace_bytes(CODE[dtype], T, V, K) > 256
    assert _lp().lp_distill_top_workspace_bytes(CODE[dtype], T, V) > 256


def _top(x, z, K, tau=1.0):
    got = [host(g) for g in _lp().lp_top_logits(x, K, None, tau)]
    with np.errstate(invalid="ignore"):
        want = O.top_logits(z, K, None, tau)
    assert np.array_equal(got[0], want[0])
    for g, w in zip(got[1:], want[1:]):
        close(g, w, tol_log(w, 2))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [70001, 200003])
@pytest.mark.parametrize("K", [1, 40, 256])
def test_top_special_values(dtype, V, K):
    """NaN, +inf and -inf in a first, an inner and a last slice, zeros of both signs, whole slices without a value."""
    rng = np.random.default_rng(V + K)
    z = rng.normal(0, 3, (13, V))
    z[0, 7] = z[1, V // 2] = z[2, V - 1] = np.nan
    z[3, 7] = z[4, V // 2] = z[5, V - 1] = np.inf
    z[6] = -np.inf
    z[7, ::2] = -np.inf
    z[8] = np.where(rng.random(V) < 0.5, -0.0, 0.0)
    z[9, :V - 3] = -np.inf
    z[10, 3:] = -np.inf
    z[11] = -np.inf
    z[11, V // 2] = 1.0
    z[12, [5, V // 3, V // 2, V - 2]] = 40.0
    bits = to_bits(z, dtype)
    _cut(dtype, 13, V, K)
    _top(dev_rows(bits, dtype), O.widen(bits, dtype), K)


@pytest.mark.parametrize("dtype", DTYPES)
def test_distillation_special_values(dtype):
    """The same through the loss: entries, NaN and infinities in other slices than each other."""
    torch, lp = _torch(), _lp()
    V, K, T = 70001, 12, 11
    rng = np.random.default_rng(4)
    z0 = rng.normal(0, 3, (T, V))
    ids, lpk, rest = lists(rng, O.widen(to_bits(z0, dtype), dtype), K, 1.0, pad=False)
    low = {"bf16": -3.3e38, "fp16": -65504.0, "fp32": -3.4e38}[dtype]
    z0[0, 50], z0[1, V - 1], z0[2] = np.nan, np.inf, -np.inf
    z0[3, ids[3, 2]] = -np.inf                                       # the teacher has mass there
    z0[4] = np.where(np.isin(np.arange(V), ids[4]), z0[4], -np.inf)  # no weight outside the list
    z0[5] = np.where(np.isin(np.arange(V), ids[5]), -np.inf, z0[5])  # none in it
    z0[6, 100:V - 100] = low
    z0[7, ids[7, 0]] = np.nan
    z0[8, :V // 2] = -np.inf
    ids[8] = V // 2 + 1 + np.arange(K) * 5
    lpk[9, 1] = np.nan
    ids[10, :4], ids[10, 4:] = V - 1, 0                              # both ends, each several times
    bits = to_bits(z0, dtype)
    z = O.widen(bits, dtype)
    _cut(dtype, T, V, K)
    x, a = dev_rows(bits, dtype), [to_dev(t) for t in (ids, lpk, rest)]
    with np.errstate(invalid="ignore", over="ignore"):
        want = O.distill_top(z, ids, lpk, rest, None, 1.0)
    got = [host(t) for t in lp.lp_distill_top(x, *a)]
    assert np.isnan(got[0][[0, 1, 2, 7, 9]]).all() and np.isnan(got[1][[0, 1, 7]]).all() and got[1][2] == -np.inf
    assert (got[0][[3, 4, 5]] == np.inf).all() and got[2][4] == -np.inf
    mass = np.exp(lpk.astype(np.float64)).sum(1) + np.exp(rest.astype(np.float64))
    rows = [3, 4, 5, 6, 8, 10]
    tol = 2 * SUM * (1 + mass) + 2.0 ** -24 * np.abs(np.where(np.isfinite(want[0]), want[0], 0))
    close(got[0][rows], want[0][rows], tol[rows])
    for g, w in zip(got[1:], want[1:]):
        close(g[rows + [9]], w[rows + [9]], tol_log(w[rows + [9]]))
    one = torch.ones(T, device="cuda")
    d = host(lp.lp_distill_top_backward(x, *a, None, 1.0, to_dev(got[1]), to_dev(got[2]), one).float())
    assert np.isnan(d[[0, 1]]).all() and not d[2].any()
    ref = O.distill_top_backward(z[rows], ids[rows], lpk[rows], rest[rows], None, 1.0, np.ones(len(rows)))
    close(d[rows], ref, grad_tol(z[rows], ids[rows], lpk[rows], rest[rows], 1.0, np.ones(len(rows)), ref, dtype))



@pytest.mark.parametrize("T,V,K,dtype", [(70, 66497, 20, "fp32"), (36, 123088, 20, "fp32"), (56, 164859, 10, "fp16"),
                                         (68, 135830, 43, "bf16"), (27, 82045, 100, "fp32"), (18, 99214, 150, "bf16"),
                                         (1, 122913, 65, "fp32"), (35, 159221, 225, "fp32")])
def test_short_last_slices(T, V, K, dtype):
    """Sizes at which a first cut leaves a last slice too short to stream (all but the last of these, some of them
    several times): the row is cut into fewer, longer ones."""
    _cut(dtype, T, V, K)
    bits, z = peaked(np.random.default_rng(V), T, V, dtype)
    z[:, -1] = 25.0  # the row's end takes part in the list
    bits[:, -1] = to_bits(z[:, -1], dtype)
    _top(dev_rows(bits, dtype), z, K)


def _calls(seed):
    """Inputs of cut rows, and a function that makes the calls on them."""
    torch, lp = _torch(), _lp()
    rng = np.random.default_rng(seed)
    T, V, K, B, W = 6, 70001, 20, 2, 3
    teacher = to_dev_bits(peaked(rng, T, V, "bf16")[0], "bf16")
    student = to_dev_bits(peaked(rng, T, V, "bf16")[0], "bf16")
    mask = to_dev((np.arange(T) != seed % T).astype(np.uint8))
    g = to_dev(rng.normal(0, 1, T).astype(np.float32))
    scores = to_dev(-rng.uniform(0, 9, (B, W)).astype(np.float32))
    _cut("bf16", T, V, K)

    def step(stream=None, workspace=None):
        k, w = dict(stream=stream), dict(stream=stream, workspace=workspace)
        top = lp.lp_top_logits(teacher, K, mask, 1.2, **w)
        many = lp.lp_top_logits(teacher, 200, mask, 1.2, **w)
        f = lp.lp_distill_top(student, *top[:3], mask, 1.2, **w)
        d = lp.lp_distill_top_backward(student, *top[:3], mask, 1.2, f[1], f[2], g, **k)
        beams = lp.lp_beam_select(student, scores, 12, None, 3, 0.8, **w)
        return [*top, *many, *f, d, *beams]

    return [teacher, student, mask, g, scores], step


def _equal(p, q):
    torch = _torch()
    return all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(p, q))


def test_captured_and_replayed():
    """Two graphs, each with workspaces of its own, replayed in turn with other inputs and eager calls between."""
    torch = _torch()
    inputs, step = _calls(2)
    others = [_calls(20 + k)[0] for k in range(3)]
    step()
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            got.append(step())
    for k, other in enumerate(others + others[:1]):
        for a, b in zip(inputs, other):
            a.copy_(b)
        eager = step()
        torch.cuda.synchronize()
        for n in ((0, 1) if k % 2 else (1, 0)):
            graphs[n].replay()
            again = step()
            torch.cuda.synchronize()
            assert _equal(got[n], eager) and _equal(again, eager), (k, n)


def test_two_streams_at_once():
    torch = _torch()
    both = [_calls(4), _calls(5)]
    kept = [[a.clone() for a in inputs] for inputs, _ in both]
    alone = [step() for _, step in both]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [step(s) for (_, step), s in zip(both, streams)]
        torch.cuda.synchronize()
        assert all(_equal(p, q) for p, q in zip(got, alone))
    assert all(_equal(p, q) for p, (q, _) in zip(kept, both))


def test_one_workspace_for_calls_in_turn():
    """What an earlier call of another kind or size left in a workspace changes nothing, unscored rows among them."""
    torch = _torch()
    _, step = _calls(6)
    want = step()
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    for fill in (0, 255, 0x7f):
        ws.fill_(fill)
        assert _equal(step(workspace=ws), want)


def test_a_workspace_of_just_the_size():
    """What lies behind the bytes that a call asks for is left alone."""
    torch, lp = _torch(), _lp()
    (teacher, student, mask, _, scores), _ = _calls(7)
    top = lp.lp_top_logits(teacher, 20, mask, 1.2)
    T, V = teacher.shape
    for need, call in (
            (lp.lp_top_workspace_bytes(0, T, V, 200), lambda w: lp.lp_top_logits(teacher, 200, mask, workspace=w)),
            (lp.lp_distill_top_workspace_bytes(0, T, V), lambda w: lp.lp_distill_top(student, *top[:3], mask, workspace=w)),
            (lp.lp_beam_workspace_bytes(0, 2, 3, V, 12), lambda w: lp.lp_beam_select(student, scores, 12, workspace=w))):
        assert need > 256
        ws = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
        assert _equal(call(ws[:need]), call(None))
        assert bool((ws[need:] == 0x5a).all())
        with pytest.raises(ValueError, match="too small"):
            call(ws[:need - 1])
