"""GPU parity of the embedding lookup and its weight gradient.

Tolerances.  Lookup: one fp32 product and one rounding, eps/2 + 2^-24 relative
(plus half the smallest fp16 subnormal).  Gradient: a sum of n fp32 terms in
any fixed order is off by at most n 2^-24 sum |g| scale, plus two roundings
(scale, and the addition to the old value): (n + 2) 2^-24 (|base| + scale sum |g|)."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.helpers import host, to_dev, to_dev_bits
from tests.rules_cases import DTYPES, EPS, to_bits

pytestmark = pytest.mark.gpu


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def _torch():
    import torch
    return torch


def _dev(bits, dtype):
    return to_dev(bits) if dtype == "fp32" else to_dev_bits(bits, dtype)


def _case(N, h, V, dtype, seed, skew=False, extra=0):
    rng = np.random.default_rng(seed)
    W = to_bits(rng.normal(0, 1, (V, h + extra)), dtype)
    G = to_bits(rng.normal(0, 1, (N, h + extra)), dtype)
    tok = rng.integers(0, V, N).astype(np.int64)
    if skew and N:
        tok[rng.random(N) < 0.6] = V // 2  # one token is most of the text
    bad = rng.random(N) < 0.05
    tok[bad] = rng.choice([-1, V, -2**63, 2**63 - 1, 2**32], int(bad.sum()))
    return W, G, tok


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,h,V,extra", [(1, 1, 1, 0), (1, 5120, 1000, 0), (37, 7, 11, 0), (64, 256, 1024, 0),
                                         (130, 513, 77, 0), (33, 1031, 300, 3), (9, 520, 50, 8), (5, 64, 5, 1)])
def test_lookup(dtype, N, h, V, extra):
    torch = _torch()
    W, _, tok = _case(N, h, V, dtype, N + h, extra=extra)
    scale = float(np.float32(np.sqrt(h)))
    w = _dev(W, dtype)[:, extra:]
    want = O.embedding(O.widen(W, dtype)[:, extra:], tok, scale)
    got = host(_lp().lp_embedding(w, to_dev(tok), scale).float())
    tol = (EPS[dtype] / 2 + 2.0 ** -23) * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(got - want) <= tol)
    known = (tok >= 0) & (tok < V)
    assert np.all(got[~known] == 0)
    buf = torch.full((N, h + 9), 5.0, dtype=w.dtype, device="cuda")
    _lp().lp_embedding(w, to_dev(tok), scale, out=buf[:, 4:4 + h])
    b = host(buf.float())
    assert np.array_equal(b[:, 4:4 + h], got) and np.all(b[:, :4] == 5) and np.all(b[:, 4 + h:] == 5)


def test_lookup_keeps_the_tokens_shape_and_special_values():
    torch = _torch()
    w = torch.randn(10, 24, device="cuda").bfloat16()
    w[3, 5], w[4, 6] = float("nan"), float("-inf")
    tok = torch.tensor([[3, 4, 1], [9, 10, 0]], device="cuda")
    out = _lp().lp_embedding(w, tok)
    assert out.shape == (2, 3, 24)
    assert torch.equal(out[0].view(torch.int16), w[[3, 4, 1]].view(torch.int16)) and not out[1, 1].any()


def _check_grad(got, G, tok, V, scale, base=None):
    want = O.embedding_backward(G, tok, V, scale, base)
    mag = O.embedding_backward(np.abs(G), tok, V, abs(scale), None if base is None else np.abs(base))
    known = tok[(tok >= 0) & (tok < V)]
    n = np.bincount(known, minlength=V)[:, None] if known.size else np.zeros((V, 1))
    assert np.all(np.abs(got - want) <= (n + 2) * 2.0 ** -24 * mag)
    return n[:, 0] > 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,h,V,skew,extra", [
    (1, 1, 1, False, 0), (1, 40, 300, False, 0), (64, 256, 1024, False, 0), (63, 7, 5, True, 0), (65, 8, 2, True, 0),
    (1000, 1031, 300, True, 0), (256, 40, 60, True, 0), (255, 12, 70000, False, 1), (300, 2, 9000, False, 0),
    (257, 64, 70000, False, 0), (4096, 24, 500, True, 0), (4097, 24, 500, True, 0),
    (6000, 33, 66000, False, 3), (9001, 16, 3, True, 8), (20000, 8, 257, True, 0), (5000, 4, 17000000, False, 0)])
def test_gradient(dtype, N, h, V, skew, extra):
    torch = _torch()
    if V > 10**6 and dtype != "bf16":
        pytest.skip("one type is enough for the four-pass sort of a wide vocabulary")
    _, G, tok = _case(N, h, 1 if V > 10**6 else V, dtype, N + h, skew, extra)
    if V > 10**6:
        tok = np.random.default_rng(1).integers(V - 3000, V, N).astype(np.int64)
    g = _dev(G, dtype)[:, extra:]
    G64 = O.widen(G, dtype)[:, extra:]
    t = to_dev(tok)
    lp = _lp()
    out = torch.full((V, h), float("nan"), device="cuda")  # overwritten whole
    lp.lp_embedding_backward(g, t, V, 1.5, grad_weight=out)
    if V > 10**6:
        assert not out[:V - 3000].any()
        out, tok, V = out[V - 3000:], tok - (V - 3000), 3000
        _check_grad(host(out), G64, tok, V, 1.5)
        return
    first = host(out)
    _check_grad(first, G64, tok, V, 1.5)
    lp.lp_embedding_backward(g, t, V, 1.5, grad_weight=out)
    assert np.array_equal(first, host(out))  # the same bits again
    base = np.random.default_rng(3).normal(0, 1, (V, h)).astype(np.float32)
    acc = to_dev(base)
    lp.lp_embedding_backward(g, t, V, -0.25, grad_weight=acc, accumulate=True)
    there = _check_grad(host(acc), G64, tok, V, -0.25, base)
    assert np.array_equal(host(acc)[~there], base[~there])


def test_gradient_leaves_rows_of_absent_tokens_unread():
    """NaN in rows that no token names stays, and does not spread."""
    torch = _torch()
    acc = torch.full((9, 8), float("nan"), device="cuda")
    acc[4] = 1.0
    g = torch.ones(3, 8, device="cuda")
    _lp().lp_embedding_backward(g, torch.tensor([4, -1, 4], device="cuda"), 9, 2.0, grad_weight=acc, accumulate=True)
    assert torch.equal(acc[4], torch.full((8,), 5.0, device="cuda")) and torch.isnan(acc[[0, 1, 2, 3, 5, 6, 7, 8]]).all()


@pytest.mark.parametrize("N", [64, 5000])
def test_all_tokens_equal_or_unknown(N):
    torch = _torch()
    g = torch.randn(N, 40, device="cuda")
    lp = _lp()
    for v in (0, 6):
        out = lp.lp_embedding_backward(g, torch.full((N,), v, device="cuda"), 7, 1.0)
        want = g.double().sum(0)
        assert (out[v].double() - want).abs().max() <= N * 2.0 ** -24 * g.abs().sum(0).max()
        out[v] = 0
        assert not out.any()
    assert not lp.lp_embedding_backward(g, torch.full((N,), 7, device="cuda"), 7, 1.0).any()


def test_empty():
    torch = _torch()
    lp = _lp()
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert lp.lp_embedding(torch.ones(3, 5, device="cuda"), t).shape == (0, 5)
    g = torch.zeros(0, 5, device="cuda")
    assert not lp.lp_embedding_backward(g, t, 3).any()
    base = torch.ones(3, 5, device="cuda")
    lp.lp_embedding_backward(g, t, 3, grad_weight=base, accumulate=True)
    assert bool((base == 1).all())


def test_offsets_past_32_bits():
    """Rows past 2^32 bytes of the weight, the gradient of the output and dW."""
    torch = _torch()
    lp = _lp()
    V, h = 300000, 8192  # 4.9 GB in bf16, 9.8 GB of dW
    w = torch.zeros((V, h), dtype=torch.bfloat16, device="cuda")
    w[-1] = torch.arange(h, device="cuda") % 100
    tok = torch.tensor([V - 1, 5, V - 1], device="cuda")
    out = lp.lp_embedding(w, tok, 2.0)
    assert torch.equal(out[0], w[-1] * 2) and torch.equal(out[2], w[-1] * 2) and not out[1].any()
    d = lp.lp_embedding_backward(out, tok, V, 1.0)
    assert torch.equal(d[-1], w[-1].float() * 4) and not d[:-1].any()
    big = torch.arange(V, device="cuda")
    big[-1] = 0
    d = lp.lp_embedding_backward(w, big, 4, 1.0)  # the last row's position lies past 2^32 bytes
    assert torch.equal(d[0], w[-1].float()) and not d[1:].any()


def test_tied_head_step():
    """Lookup, fused head forward and backward, and the embedding's gradient
    added to the head's: the gradient of the whole with respect to the tied
    matrix, against fp64 and against differences."""
    torch = _torch()
    lp = _lp()
    rng = np.random.default_rng(21)
    N, h, V, scale, tau = 96, 64, 200, 1.25, 0.9
    Wb = to_bits(rng.normal(0, 0.3, (V, h)), "bf16")
    W = O.widen(Wb, "bf16")
    tok = rng.integers(0, 12, N).astype(np.int64)
    y = rng.integers(0, V, N).astype(np.int64)
    g = rng.normal(0, 1, N).astype(np.float32)
    w, t, yd = to_dev_bits(Wb, "bf16"), to_dev(tok), to_dev(y)
    hid = lp.lp_embedding(w, t, scale)
    _, H, lse = lp.lp_lm_head_logprobs_entropy(hid, w, yd, None, tau, 32)
    dH, dW = lp.lp_lm_head_logprobs_entropy_backward(hid, w, yd, None, tau, 32, lse, H, to_dev(g))
    head = dW.clone()
    lp.lp_embedding_backward(dH, t, V, scale, grad_weight=dW, accumulate=True)
    # exactly the head's gradient plus the scattered hidden gradient
    _check_grad(host(dW), host(dH).astype(np.float64), tok, V, scale, host(head).astype(np.float64))

    def loss(M):
        x = O.embedding(M, tok, scale)
        return O.lm_head_loss(x, M, y, None, tau, g, None)

    d = rng.normal(0, 1, (V, h))
    e = 1e-6
    slope = (loss(W + e * d) - loss(W - e * d)) / (2 * e)
    # dZ, hidden rows and their product are bf16 inside the head's backward:
    # each factor is off by 2^-9 relative, three of them, on sums of mixed sign
    got = float((host(dW).astype(np.float64) * d).sum())
    assert abs(got - slope) <= 3 * 2.0 ** -8 * float((np.abs(host(dW)) * np.abs(d)).sum())


def test_captured_and_on_another_stream():
    torch = _torch()
    lp = _lp()
    N, h, V = 5000, 72, 900
    w = torch.randn(V, h, device="cuda").bfloat16()
    tok = torch.randint(0, 40, (N,), device="cuda")
    g = torch.randn(N, h, device="cuda").bfloat16()
    acc = torch.zeros(V, h, device="cuda")

    def step(stream=None):
        a = lp.lp_embedding(w, tok, 1.5, stream=stream)
        b = lp.lp_embedding_backward(g, tok, V, 1.5, stream=stream)
        c = lp.lp_embedding_backward(g[:100], tok[:100], V, 1.5, stream=stream)
        return [a, b, c]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
        lp.lp_embedding_backward(g, tok, V, 1.0, grad_weight=acc, accumulate=True)
    acc.zero_()
    want_acc = torch.zeros_like(acc)
    side = torch.cuda.Stream()
    for k in range(5):
        tok.copy_(torch.randint(-1, 40 + 200 * k, (N,), device="cuda"))
        g.normal_()
        eager = step()
        lp.lp_embedding_backward(g, tok, V, 1.0, grad_weight=want_acc, accumulate=True)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, eager)) and torch.equal(acc, want_acc), k
        other = step(side)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(other, eager)), k


@pytest.mark.parametrize("N,h,V", [(5, 6, 9), (300, 516, 70), (5000, 30, 400)])
def test_a_weight_gradient_off_the_16_byte_grid(N, h, V):
    """dW may start at any fp32: its neighbours stay."""
    torch = _torch()
    lp = _lp()
    g = torch.randn(N, h, device="cuda")
    t = torch.randint(0, V, (N,), device="cuda")
    want = lp.lp_embedding_backward(g, t, V, 2.0)
    buf = torch.full((V * h + 8,), 3.0, device="cuda")
    for off in (1, 2, 3):
        dw = buf[off:off + V * h].view(V, h)
        lp.lp_embedding_backward(g, t, V, 2.0, grad_weight=dw)
        assert torch.equal(dw, want) and bool((buf[:off] == 3).all()) and bool((buf[off + V * h:] == 3).all())
        lp.lp_embedding_backward(g, t, V, 2.0, grad_weight=dw, accumulate=True)
        assert torch.equal(dw, want + want)
        buf.fill_(3.0)


def test_inputs_unchanged_and_two_streams_at_once():
    """No call writes its inputs, and calls that overlap on two streams, each
    with its own outputs and workspace, agree with the calls made alone."""
    torch = _torch()
    lp = _lp()
    w = torch.randn(3000, 264, device="cuda").bfloat16()
    gs = [torch.randn(6000, 264, device="cuda").bfloat16() for _ in range(2)]
    ts = [torch.randint(-2, 3002, (6000,), device="cuda") for _ in range(2)]
    kept = [x.clone() for x in (w, *gs, *ts)]
    alone = [(lp.lp_embedding(w, t, 0.5), lp.lp_embedding_backward(g, t, 3000, 0.5)) for g, t in zip(gs, ts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [(lp.lp_embedding(w, t, 0.5, stream=s), lp.lp_embedding_backward(g, t, 3000, 0.5, stream=s))
               for g, t, s in zip(gs, ts, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for p, q in zip(got, alone) for a, b in zip(p, q))
    assert all(torch.equal(a, b) for a, b in zip(kept, (w, *gs, *ts)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,h,V,off", [(100, 768, 500, 1), (200, 1025, 900, 2), (300, 1026, 4000, 3), (3000, 771, 900, 1),
                                       (5000, 1036, 700, 5), (4500, 1541, 3000, 6), (700, 2047, 130, 31)])
def test_long_rows_on_any_boundary(dtype, N, h, V, off):
    """Rows off the 16-byte grid and of a broken last vector; stretches of absent rows from any boundary on."""
    torch = _torch()
    lp = _lp()
    _, G, tok = _case(N, h, V, dtype, N + h, True, 3)
    tok[tok > V // 2] = V // 2  # the upper half of the vocabulary is one stretch
    g, G64, t = _dev(G, dtype)[:, 3:], O.widen(G, dtype)[:, 3:], to_dev(tok)
    whole = torch.full((off + V * h + 40,), 7.0, device="cuda")
    out = whole[off:off + V * h].view(V, h)
    lp.lp_embedding_backward(g, t, V, 1.5, grad_weight=out)
    _check_grad(host(out), G64, tok, V, 1.5)
    assert (whole[:off] == 7).all() and (whole[off + V * h:] == 7).all()
    base = np.random.default_rng(4).normal(0, 1, (V, h)).astype(np.float32)
    out.copy_(to_dev(base))
    lp.lp_embedding_backward(g, t, V, -0.25, grad_weight=out, accumulate=True)
    there = _check_grad(host(out), G64, tok, V, -0.25, base)
    assert np.array_equal(host(out)[~there], base[~there])
    assert (whole[:off] == 7).all() and (whole[off + V * h:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("h", [1, 9, 1031, 2050])
def test_lookup_of_rows_at_every_boundary(dtype, h):
    torch = _torch()
    W, _, tok = _case(70, h, 90, dtype, h, extra=8)
    for a, b in ((0, 1), (1, 0), (3, 6), (7, 2)):
        w = _dev(W, dtype)[:, a:a + h]
        want = O.embedding(O.widen(W, dtype)[:, a:a + h], tok, 1.0)  # a scale of 1 rounds nothing
        buf = torch.full((70, h + 9), 5.0, dtype=w.dtype, device="cuda")
        _lp().lp_embedding(w, to_dev(tok), 1.0, out=buf[:, b:b + h])
        got = host(buf.float())
        assert np.array_equal(got[:, b:b + h], want) and np.all(got[:, :b] == 5) and np.all(got[:, b + h:] == 5)
