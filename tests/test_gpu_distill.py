"""GPU parity of distillation from a teacher's top logits against the fp64 oracle, its gradient also against differences of the
loss that the kernel itself gives."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.choose_cases import SUM, close, dev_rows, grad_tol, lists, peaked, tol_log
from tests.helpers import host, to_dev
from tests.rules_cases import DTYPES, to_bits

pytestmark = pytest.mark.gpu


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def check(x, z, ids, lpk, rest, tau, mask, dtype, grad=True, out=None):
    """Loss and gradient of device rows x against the oracle on their fp64 values z."""
    lp = _lp()
    T = z.shape[0]
    d = lambda a: None if a is None else to_dev(a)  # noqa: E731
    with np.errstate(invalid="ignore", over="ignore"):
        want = O.distill_top(z, ids, lpk, rest, mask, tau)
    got = lp.lp_distill_top(x, d(ids), d(lpk), d(rest), d(mask), tau)
    mass = np.where((ids >= 0) & (ids < z.shape[1]), np.exp(lpk.astype(np.float64)), 0).sum(1)
    if rest is not None:
        mass = mass + np.exp(rest.astype(np.float64))
    close(host(got[0]), want[0], 2 * SUM * (1 + mass) + 2.0 ** -24 * np.abs(np.where(np.isfinite(want[0]), want[0], 0)))
    for g, w in zip(got[1:], want[1:]):
        close(host(g), w, tol_log(w))
    if not grad:
        return got
    gl = np.linspace(-1, 1, T).astype(np.float32) + np.float32(0.01)
    want = O.distill_top_backward(z, ids, lpk, rest, mask, tau, gl)
    d = lp.lp_distill_top_backward(x, d(ids), d(lpk), d(rest), d(mask), tau, got[1], got[2], to_dev(gl), grad_logits=out)
    tol = grad_tol(z, ids, lpk, rest, tau, gl, want, dtype)
    close(host(d.float()), want, tol)
    return got, d


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("with_rest", [True, False])
@pytest.mark.parametrize("T,V,K", [
    (1, 1, 1), (2, 3, 2), (3, 9, 5), (37, 1000, 17), (5, 4099, 64), (2, 20011, 256), (1, 151936, 64), (800, 5003, 20),
    (770, 20003, 64), (3, 131075, 33)])
def test_shapes(dtype, with_rest, T, V, K):
    import torch
    rng = np.random.default_rng(T + V + K)
    bits, z = peaked(rng, T, V, dtype, extra=5)
    ids, lpk, rest = lists(rng, z, K, 1.3)
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    mask[0] = 1
    x = dev_rows(bits, dtype)[:, :V]
    out = torch.full((T, V + 3), 7.0, dtype=x.dtype, device="cuda")  # gradients off the 16-byte grid
    _, d = check(x, z, ids, lpk, rest if with_rest else None, 1.3, mask, dtype, out=out[:, 1:1 + V])
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 1 + V:] == 7).all())
    assert not host(d.float())[mask == 0].any()
    # a contiguous call gives the same bits
    a = [to_dev(t) for t in (ids, lpk, rest)]
    if not with_rest:
        a[2] = None
    y = x.contiguous()
    f = [_lp().lp_distill_top(v, *a, to_dev(mask), 1.3) for v in (x, y)]
    assert all(torch.equal(p, q) for p, q in zip(*f))
    g = torch.ones(T, device="cuda")
    e = [_lp().lp_distill_top_backward(v, *a, to_dev(mask), 1.3, f[0][1], f[0][2], g) for v in (x, y)]
    assert torch.equal(e[0], e[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_lists(dtype):
    """All of a vocabulary, one vector of it, one id many times, padding alone, ids at the ends, neighbours."""
    V = 200
    rng = np.random.default_rng(9)
    bits, z = peaked(rng, 7, V, dtype)
    ids = np.zeros((7, 200), dtype=np.int64)
    lpk = np.full((7, 200), np.log(1 / 300), dtype=np.float32)
    ids[0] = rng.permutation(V)
    ids[1] = np.arange(200) % 8 + 64
    ids[2] = 131
    ids[3] = -5
    ids[4] = np.where(np.arange(200) < 100, 0, V - 1)
    ids[5] = np.arange(200) // 2
    ids[6] = rng.integers(-3, V + 3, 200)
    rest = np.full(7, np.log(0.2), dtype=np.float32)
    rest[0] = -np.inf
    for r in (rest, None):
        check(dev_rows(bits, dtype), z, ids, lpk, r, 0.9, None, dtype)
    # mass outside the list where the student has none
    rest[0] = -3.0
    loss = check(dev_rows(bits, dtype), z, ids, lpk, rest, 0.9, None, dtype, grad=False)[0]
    assert host(loss)[0] == np.inf and np.isfinite(host(loss)[1:]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_special_values(dtype):
    import torch
    V, K = 3001, 12
    rng = np.random.default_rng(4)
    z0 = rng.normal(0, 3, (9, V))
    bits = to_bits(z0, dtype)
    ids, lpk, rest = lists(rng, O.widen(bits, dtype), K, 1.0, pad=False)
    low = {"bf16": -3.3e38, "fp16": -65504.0, "fp32": -3.4e38}[dtype]
    z0[0, 50], z0[1, V - 1], z0[2] = np.nan, np.inf, -np.inf
    z0[3, ids[3, 2]] = -np.inf                            # the teacher has mass there
    z0[4] = np.where(np.isin(np.arange(V), ids[4]), z0[4], -np.inf)  # no weight outside the list
    z0[5] = np.where(np.isin(np.arange(V), ids[5]), -np.inf, z0[5])  # none in it
    z0[6, 100:2900] = low
    z0[7] = low
    lpk[8, 1] = np.nan
    bits = to_bits(z0, dtype)
    z = O.widen(bits, dtype)
    x = dev_rows(bits, dtype)
    with np.errstate(invalid="ignore", over="ignore"):
        want = O.distill_top(z, ids, lpk, rest, None, 1.0)
    got = [host(t) for t in _lp().lp_distill_top(x, to_dev(ids), to_dev(lpk), to_dev(rest))]
    assert np.isnan(got[0][[0, 1, 2, 8]]).all() and np.isnan(got[1][[0, 1]]).all() and got[1][2] == -np.inf
    assert got[0][3] == np.inf and got[0][4] == np.inf and got[0][5] == np.inf
    assert np.isfinite(got[0][6])
    for t in (3, 4, 5, 6, 8):
        for g, w in zip(got[1:], want[1:]):
            close(g[t:t + 1], w[t:t + 1], tol_log(w[t:t + 1]))
    g = torch.ones(9, device="cuda")
    d = host(_lp().lp_distill_top_backward(x, to_dev(ids), to_dev(lpk), to_dev(rest), None, 1.0, to_dev(got[1]), to_dev(got[2]), g).float())
    assert np.isnan(d[0]).all() and np.isnan(d[1]).all() and not d[2].any() and np.isnan(d[8]).any()
    with np.errstate(invalid="ignore", over="ignore"):
        ref = O.distill_top_backward(z, ids, lpk, rest, None, 1.0, np.ones(9))
        tol = grad_tol(z, ids, lpk, rest, 1.0, np.ones(9), ref, dtype)
    for t in (3, 4, 5, 6):
        close(d[t], ref[t], tol[t])
    # a student without any weight outside, and a teacher without any: that term is 0
    rest[4] = -np.inf
    loss = host(_lp().lp_distill_top(x, to_dev(ids), to_dev(lpk), to_dev(rest))[0])
    want = O.distill_top(z[4:5], ids[4:5], lpk[4:5], rest[4:5], None, 1.0)[0]
    close(loss[4:5], want, 1e-4)


def test_student_equal_to_its_teacher():
    """A student that is its teacher: loss 0 and gradient 0 up to roundings of the masses."""
    import torch
    lp = _lp()
    z = torch.randn(40, 30011, device="cuda") * 3
    ids, p, rest, lse = lp.lp_top_logits(z, 64)
    loss, a, b = lp.lp_distill_top(z, ids, p, rest)
    assert loss.abs().max() <= 4 * SUM and (a - lse).abs().max() <= 2 * SUM + 1e-6
    assert (b - (rest + lse)).abs().max() <= 4 * SUM + 1e-5
    d = lp.lp_distill_top_backward(z, ids, p, rest, None, 1.0, a, b, torch.ones(40, device="cuda"))
    q = torch.softmax(z.double(), 1)
    assert (d.double().abs() <= q * 2e-4 + 1e-9).all()


def test_gradient_against_differences():
    """Directional differences of the kernel's own loss in fp32 at a step where its rounding (1e-6 of values near 1) and the
    third derivative (step^2 / 6) are both below 1e-4 of the slope's scale."""
    import torch
    lp = _lp()
    torch.manual_seed(1)
    T, V, K = 16, 501, 20
    z = torch.randn(T, V, device="cuda")
    t = torch.randn(T, V, device="cuda")
    ids, p, rest, _ = lp.lp_top_logits(t, K)
    g = torch.linspace(0.5, 1.5, T, device="cuda")
    _, a, b = lp.lp_distill_top(z, ids, p, rest, None, 0.8)
    d = lp.lp_distill_top_backward(z, ids, p, rest, None, 0.8, a, b, g)
    for seed in range(4):
        torch.manual_seed(seed)
        v = torch.randn(T, V, device="cuda")
        f = lambda s: (lp.lp_distill_top(z + s * v, ids, p, rest, None, 0.8)[0].double() * g.double()).sum(0)  # noqa: E731
        h = 2e-2
        slope = (f(h) - f(-h)) / (2 * h)
        want = (d.double() * v.double()).sum()
        assert abs(slope - want) <= 2e-3 * max(1.0, abs(float(want)))


def test_empty_and_many_rows():
    import torch
    lp = _lp()
    none = lp.lp_distill_top(torch.zeros(0, 9, device="cuda"), torch.zeros(0, 3, dtype=torch.int64, device="cuda"),
                             torch.zeros(0, 3, device="cuda"))
    assert none[0].numel() == 0
    T = (1 << 22) + 9001
    z = torch.randn(T, 3, device="cuda")
    ids = torch.randint(-1, 4, (T, 1), device="cuda")
    p = torch.full((T, 1), -0.5, device="cuda")
    loss, lse, lse_rest = lp.lp_distill_top(z, ids, p)
    logq = torch.log_softmax(z.double(), 1)
    ok = (ids >= 0) & (ids < 3)
    want = torch.where(ok, np.exp(-0.5) * (-0.5 - logq.gather(1, ids.clamp(0, 2))), 0.0)[:, 0]
    assert (loss.double() - want).abs().max() <= 1e-5
    d = lp.lp_distill_top_backward(z, ids, p, None, None, 1.0, lse, lse_rest, torch.ones(T, device="cuda"))
    ref = np.exp(-0.5) * logq.exp()
    ref.scatter_add_(1, ids.clamp(0, 2), torch.where(ok, -np.exp(-0.5), 0.0).double())
    assert (d.double() - torch.where(ok, ref, 0.0)).abs().max() <= 1e-5


def test_a_vocabulary_at_the_limit():
    import torch
    V = 1 << 30
    z = torch.zeros(1, V, dtype=torch.bfloat16, device="cuda")
    z[0, V - 1] = 20.0
    ids = torch.tensor([[V - 1, 5, 1 << 29]], device="cuda")
    p = torch.log(torch.tensor([[0.5, 0.2, 0.1]], device="cuda"))
    rest = torch.log(torch.tensor([0.2], device="cuda"))
    loss, lse, lse_rest = _lp().lp_distill_top(z, ids, p, rest)
    s = np.exp(20.0) + V - 1
    q = np.array([np.exp(20.0) / s, 1 / s, 1 / s])
    m = np.array([0.5, 0.2, 0.1])
    want = (m * np.log(m / q)).sum() + 0.2 * np.log(0.2 / ((V - 3) / s))
    close(host(loss), [want], 1e-4)
    d = _lp().lp_distill_top_backward(z, ids, p, rest, None, 1.0, lse, lse_rest, torch.full((1,), 1e6, device="cuda"))
    got = host(d[0, [V - 1, 5, 1 << 29, 6, V - 2, (1 << 29) + 1]].float())
    other = (1 / s) - 0.2 / (V - 3)
    ref = 1e6 * np.array([q[0] - 0.5, q[1] - 0.2, q[2] - 0.1, other, other, other])
    close(got, ref, 2.0 ** -8 * np.abs(ref) + 1e-4 * np.abs(ref))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V", [(900, 12007), (3, 70001)])
def test_rests_and_peaks_anywhere(dtype, T, V):
    """Values far above and far below the first ones that a lane reads, in the list and outside it."""
    rng = np.random.default_rng(6)
    K = 9
    z = rng.normal(0, 1, (6, V))
    z[0, V // 3:] += 100.0
    z[1, V - 2] += 250.0
    z[2, :4000] = -np.inf
    z[3, 64:] -= 180.0
    z[4, ::2] -= 240.0
    z[5, 77] = 400.0
    bits = to_bits(z, dtype)
    z = O.widen(bits, dtype)
    ids, lpk, rest = lists(rng, z, K, 1.0)
    rows = min(T, 6)
    want = O.distill_top(z[:rows], ids[:rows], lpk[:rows], rest[:rows], None, 1.0)
    wide = lambda a: np.tile(a, (T // 6 + 1,) + (1,) * (a.ndim - 1))[:T]  # noqa: E731
    x, i, p, r = dev_rows(wide(bits), dtype), to_dev(wide(ids)), to_dev(wide(lpk)), to_dev(wide(rest))
    got = [host(g) for g in _lp().lp_distill_top(x, i, p, r)]
    mass = np.where((ids >= 0) & (ids < V), np.exp(lpk.astype(np.float64)), 0).sum(1)[:rows] + np.exp(rest.astype(np.float64))[:rows]
    # logits and log-sums of some hundreds: each is rounded where it is that large
    size = np.abs(np.where(np.isfinite(want[1]), want[1], 0)) + np.abs(np.where(np.isfinite(want[2]), want[2], 0))
    close(got[0][:rows], want[0], 2 * SUM * (1 + mass) + 2.0 ** -24 * np.abs(np.where(np.isfinite(want[0]), want[0], 0)) + mass * 2.0 ** -21 * size)
    for g, w in zip(got[1:], want[1:]):
        close(g[:rows], w, tol_log(w))
    for g in got:  # equal rows have equal bits
        assert all(np.array_equal(g[t], g[t % 6], equal_nan=True) for t in range(T))
    gl = np.linspace(0.5, 1, T).astype(np.float32)
    d = _lp().lp_distill_top_backward(x, i, p, r, None, 1.0, to_dev(got[1]), to_dev(got[2]), to_dev(gl))[:rows]
    ref = O.distill_top_backward(z[:rows], ids[:rows], lpk[:rows], rest[:rows], None, 1.0, gl[:rows])
    close(host(d.float()), ref, grad_tol(z[:rows], ids[:rows], lpk[:rows], rest[:rows], 1.0, gl[:rows], ref, dtype))
