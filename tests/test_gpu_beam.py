"""GPU parity of beam selection against the fp64 oracle (parents and tokens equal) and of the reordering of states (equal bits)."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.choose_cases import close, dev_rows, peaked, tol_log
from tests.helpers import host, to_dev
from tests.rules_cases import DTYPES, to_bits

pytestmark = pytest.mark.gpu


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def clear_scores(rng, z, B, W, N, finished, end, tau):
    """Scores so far at which no two candidates of different beams lie within 3e-5 (what two log-sums may be
    off by, 2 SUM), up to and past the N-th."""
    s = -rng.uniform(0, 12, (B, W)).astype(np.float32)
    for _ in range(200):
        sc, pa, _ = O.beam_select(z, s, N + 1, finished, end, tau)
        with np.errstate(invalid="ignore"):
            near = ((sc[:, :-1] - sc[:, 1:]) < 3e-5) & (pa[:, :-1] != pa[:, 1:]) & np.isfinite(sc[:, 1:])
        bad = near.any(1)
        if not bad.any():
            return s
        s[bad] -= rng.uniform(0, 1, (int(bad.sum()), W)).astype(np.float32)
    raise AssertionError("no such scores found")


def check(x, z, s, N, finished, end, tau):
    got = [host(g) for g in _lp().lp_beam_select(x, to_dev(s), N, None if finished is None else to_dev(finished), end, tau)]
    with np.errstate(invalid="ignore"):
        want = O.beam_select(z, s, N, finished, end, tau)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[2], want[2])
    close(got[0], want[0], tol_log(want[0]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,W,V,N", [
    (1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 7, 3), (1, 4, 20011, 8), (3, 5, 1000, 10), (64, 8, 3001, 16), (7, 10, 5003, 20),
    (2, 64, 300, 64), (1, 16, 9001, 256), (1, 1, 70001, 256), (130, 5, 2000, 5), (1, 4, 151936, 4), (70, 8, 20011, 16)])
def test_shapes(dtype, B, W, V, N):
    rng = np.random.default_rng(B + W + V + N)
    bits, z = peaked(rng, B * W, V, dtype, extra=1)
    finished = (rng.random((B, W)) < 0.2).astype(np.uint8)
    end = V // 3
    for f, tau in ((None, 1.0), (finished, 0.7)):
        s = clear_scores(rng, z, B, W, N, f, end, tau)
        if W > 2:
            s[0, 2] = -np.inf
            s[B - 1, 1] = np.nan
        with np.errstate(invalid="ignore"):
            sc, pa, _ = O.beam_select(z, s, N + 1, f, end, tau)
            near = ((sc[:, :-1] - sc[:, 1:]) < 3e-5) & (pa[:, :-1] != pa[:, 1:]) & np.isfinite(sc[:, 1:])
        assert not near.any()
        check(dev_rows(bits, dtype)[:, :V], z, s, N, f, end, tau)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [50, 9000])
def test_ties_go_to_the_lowest_beam_then_token(dtype, V):
    """Rows of the same values: every score comes up in each beam, equal to the last bit."""
    z = np.tile(np.repeat([2.0, 1.0, 0.0, -3.0], -(-V // 4))[:V][::-1], (6, 1))
    bits = to_bits(z, dtype)
    s = np.zeros((2, 3), dtype=np.float32)
    check(dev_rows(bits, dtype), O.widen(bits, dtype), s, 40, None, 0, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_that_offer_little(dtype):
    """Grammars that leave one token or none, NaN and +inf rows, every beam finished, beams that are not there."""
    V, W, N = 5000, 3, 6
    rng = np.random.default_rng(8)
    z = rng.normal(0, 3, (7 * W, V))
    z[0] = -np.inf
    z[1] = np.where(np.arange(V) == 4321, 1.0, -np.inf)
    z[2, 10:] = -np.inf
    z[3:6] = -np.inf
    z[6, 5], z[7, V - 1] = np.nan, np.inf
    z[18, 1:] = -1e4  # finite masks are candidates all the same
    bits = to_bits(z, dtype)
    s = -np.arange(21, dtype=np.float32).reshape(7, W) / 8 - np.float32(0.1)
    f = np.zeros((7, W), dtype=np.uint8)
    f[3] = 1
    s[4] = -np.inf
    s[5] = [np.inf, np.nan, -1]
    f[5, 2] = 1
    s[6, 1:] = -np.inf
    check(dev_rows(bits, dtype), O.widen(bits, dtype), s, N, f, 17, 1.0)


def test_more_requests_than_one_launch():
    import torch
    B = (1 << 21) + 5
    z = torch.randint(-40, 40, (B, 3), device="cuda").half()
    s, p, y = _lp().lp_beam_select(z, torch.zeros(B, 1, device="cuda"), 1)
    key = z.float() * 8 - torch.arange(3, device="cuda")
    assert torch.equal(y[:, 0], key.argmax(1)) and not p.any()
    assert (s[:, 0].double() - torch.log_softmax(z.double(), 1).amax(1)).abs().max() <= 1e-5


# --- states ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["uint8", "int16", "bfloat16", "int32", "float32", "int64", "complex128"])
@pytest.mark.parametrize("shape,dim,cut", [
    ((6, 1), 0, None), ((6, 5), 0, None), ((6, 1517), 0, 1000), ((3, 6, 4, 70), 1, 33), ((2, 6, 300), 1, None), ((6, 3, 9), 0, 8),
    ((5, 6), 1, None), ((1, 6, 2, 5000), 1, 4999), ((2, 3, 6, 40), 2, 16), ((6, 4100), 0, 4098)])
def test_reorder(dtype, shape, dim, cut):
    import torch
    rng = np.random.default_rng(7)
    t = torch.from_numpy(rng.integers(0, 255, (*shape, 16), dtype=np.uint8)).cuda()
    dt = getattr(torch, dtype)
    t = t.view(dt)[..., 0] if dt.itemsize == 16 else t.view(dt)[..., 0].contiguous()
    t = t.contiguous() if cut is None else t.contiguous()[..., :cut]
    bits = lambda a: a.contiguous().view(torch.uint8).cpu().numpy().reshape(*a.shape, -1)  # noqa: E731
    for par in ([[2, 0, 0], [1, 1, 2]], [[0, 1, 2], [-1, 3, 1]], [[0, 1, 2, 2, 0], [1, 1, 1, 1, 1]]):
        p = np.array(par, dtype=np.int32)
        want = O.beam_reorder(bits(t), p, dim)
        got = _lp().lp_beam_reorder(t, to_dev(p), dim=dim)
        assert np.array_equal(bits(got), want)
        # into the used part of a larger buffer, what lies behind it left as it was
        wide = list(got.shape)
        wide[-1] += 3
        buf = torch.zeros(wide, dtype=torch.uint8, device="cuda").unsqueeze(-1).expand(*wide, dt.itemsize).contiguous() + 9
        buf = buf.view(dt)[..., 0]
        if dim == len(shape) - 1:
            continue
        view = buf[..., :-3]
        _lp().lp_beam_reorder(t, to_dev(p), dim=dim, out=view)
        assert np.array_equal(bits(view), want) and bool((bits(buf[..., -3:]) == 9).all())


def test_reorder_refuses_what_overlaps():
    import torch
    lp = _lp()
    x = torch.zeros(8, 10, device="cuda")
    p = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(lp.LPError, match="overlaps"):
        lp.lp_beam_reorder(x[:4], p, out=x[:4])
    with pytest.raises(lp.LPError, match="overlaps"):
        lp.lp_beam_reorder(x[:4], p, out=x[3:7])
    with pytest.raises(lp.LPError, match="nested"):
        lp.lp_beam_reorder(x[:4], p, out=torch.zeros(1, 10, device="cuda").expand(4, 10))
    lp.lp_beam_reorder(x[:4], p, out=x[4:])


def test_reorder_past_four_gigabytes():
    import torch
    n = (1 << 31) + 4096  # bytes of a row
    x = torch.empty(3, n, dtype=torch.uint8, device="cuda")
    for k in range(3):
        x[k].fill_(k + 1)
        x[k, -1] = 77 + k
    got = _lp().lp_beam_reorder(x, torch.tensor([[2, 0, 2]], dtype=torch.int32, device="cuda"))
    for k, w in enumerate((2, 0, 2)):
        assert torch.equal(got[k], x[w])


@pytest.mark.parametrize("N", [8, 16])
def test_rows_whose_last_slice_is_shorter(N):
    rng = np.random.default_rng(N)
    B, W, V = 10, 8, 53277
    bits, z = peaked(rng, B * W, V, "fp32")
    s = clear_scores(rng, z, B, W, N, None, 0, 1.0)
    check(dev_rows(bits, "fp32"), z, s, N, None, 0, 1.0)
