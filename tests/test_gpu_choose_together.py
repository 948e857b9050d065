"""Runs of the choosing and distilling calls together, as a trainer and a decoder make them, in graphs and on streams.

Each call of a run is checked against the fp64 oracle on what the call before it
left on the device, so a tolerance covers one call and does not grow along a run."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.choose_cases import SUM, close, grad_tol, peaked, tol_log
from tests.helpers import host, to_dev, to_dev_bits

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def _fp8_head(rng, V, h):
    lp = _lp()
    w = rng.normal(0, 1, (V, h)).astype(np.float32) / np.float32(np.sqrt(h))
    w[rng.integers(0, V, 30)] *= 4
    return lp.lp_lm_head_fp8_quantize(to_dev(w).bfloat16())


def _fp8_tol(mag, h, want):
    """fp32 results of at most 16 or of many rows: sums of widened products (128 additions a block, each off by at most
    2^-23 of the magnitudes), blocks joined in fp32."""
    return (128 * 2.0 ** -23 + (-(-h // 128) + 11) * 2.0 ** -24) * mag


@pytest.mark.parametrize("T,h,V,K,tau", [(3, 512, 1500, 5, 1.0), (70, 384, 5003, 32, 1.6), (200, 272, 20011, 100, 0.8)])
def test_distillation_from_an_8_bit_teacher(T, h, V, K, tau):
    """Teacher's logits from the 8-bit head, their top and its log-probs, the student's loss and its gradient."""
    torch, lp = _torch(), _lp()
    rng = np.random.default_rng(T + V)
    q, s = _fp8_head(rng, V, h)
    x = torch.from_numpy(rng.normal(0, 1, (T, h))).cuda().bfloat16()
    t = lp.lp_lm_head_fp8_logits(x, q, s, out_dtype=torch.float32)
    x64 = host(x.double())
    want, mag = O.fp8_logits(x64, host(q.double()), host(s))
    close(host(t), want, _fp8_tol(mag, h, want))

    mask = torch.from_numpy(rng.random(T) < 0.8).cuda()
    mask[0] = True
    m = host(mask).astype(np.uint8)
    ids, logp, rest, _ = lp.lp_top_logits(t, K, mask, tau)
    ids_o, logp_o, rest_o, _ = O.top_logits(host(t).astype(np.float64), K, m, tau)
    assert np.array_equal(host(ids), ids_o)
    close(host(logp), logp_o, tol_log(logp_o, 2))
    close(host(rest), rest_o, tol_log(rest_o, 2))

    student = (t + torch.from_numpy(rng.normal(0, 0.7, (T, V))).cuda()).bfloat16()
    z = host(student.double())
    loss, lse, lse_rest = lp.lp_distill_top(student, ids, logp, rest, mask, tau)
    args = host(ids), host(logp), host(rest), m, tau
    loss_o, lse_o, lse_rest_o = O.distill_top(z, *args)
    close(host(loss), loss_o, 2 * SUM * 2 + 2.0 ** -24 * np.abs(loss_o))
    close(host(lse), lse_o, tol_log(lse_o))
    close(host(lse_rest), lse_rest_o, tol_log(lse_rest_o))
    # a teacher's whole distribution: the loss is no less than 0, and 0 where the student is the teacher
    assert bool((loss >= -2 * SUM * 2).all())
    same = lp.lp_distill_top(t, ids, logp, rest, mask, tau)[0]
    assert host(same).max() <= 4 * SUM * 2

    g = torch.full((T,), 1.0 / int(mask.sum()), device="cuda")
    d = lp.lp_distill_top_backward(student, ids, logp, rest, mask, tau, lse, lse_rest, g)
    d_o = O.distill_top_backward(z, *args, host(g))
    tol = grad_tol(z, host(ids), host(logp), host(rest), tau, host(g), d_o, "bf16")
    close(host(d.float()), d_o, tol)
    # a row's gradient sums to grad (mass - mass) = 0, up to the roundings of its entries
    assert np.all(np.abs(host(d.double()).sum(1)) <= tol.sum(1))


def test_decoding_with_beams():
    """Embedding, 8-bit head, a grammar and penalties, selection, then histories and a cache that follow their beams."""
    torch, lp = _torch(), _lp()
    rng = np.random.default_rng(8)
    B, W, V, h, L, end, tau = 3, 4, 2011, 256, 12, 7, 0.9
    q, s = _fp8_head(rng, V, h)
    emb = torch.from_numpy(rng.normal(0, 1, (V, h))).cuda().bfloat16()
    hist = torch.zeros(B * W, L, dtype=torch.int32, device="cuda")
    hist[:, 0] = to_dev(rng.integers(0, V, B).astype(np.int32)).repeat_interleave(W)
    cache = torch.zeros(2, B * W, 3, L, 16, dtype=torch.bfloat16, device="cuda")
    scores = torch.full((B, W), float("-inf"), device="cuda")
    scores[:, 0] = 0.0  # one beam a request at first
    finished = torch.zeros(B, W, dtype=torch.bool, device="cuda")
    words = np.full((B * W, -(-V // 32)), -1, dtype=np.int32)
    words[:, 3] = 0  # ids 96 .. 127 are not allowed
    words = to_dev(words)
    pen = torch.full((B * W,), 0.3, device="cuda")
    ref_hist, ref_cache = host(hist).copy(), host(cache.float()).copy()
    for k in range(1, L):
        x = lp.lp_embedding(emb, hist[:, k - 1].long(), 1.0)
        cache[:, :, :, k - 1] = x[:, :48].view(1, B * W, 3, 16)
        ref_cache[:, :, :, k - 1] = host(x[:, :48].float()).reshape(1, B * W, 3, 16)
        z = lp.lp_lm_head_fp8_logits(x, q, s, out_dtype=torch.float32)
        z = lp.lp_process_logits(z, lp.LogitRules(tokens=hist, hist_len=torch.full((B * W,), k, dtype=torch.int32, device="cuda"),
                                                  presence=pen, allowed=words))
        z64, sc, fin = host(z).astype(np.float64), host(scores), host(finished)
        assert np.isneginf(z64[:, 96:128]).all()
        new, parents, tokens = lp.lp_beam_select(z, scores, None, finished, end, tau)
        # scores in order and right for the candidates that were taken; no candidate twice; none better left out
        with np.errstate(invalid="ignore"):
            best, _, _ = O.beam_select(z64, sc, W, fin, end, tau)
            logp = O.log_softmax(O.tempered(z64, tau))
        close(host(new), best, tol_log(best))
        pa, to = host(parents), host(tokens)
        for b in range(B):
            taken = set()
            for n in range(W):
                p, t = int(pa[b, n]), int(to[b, n])
                if fin[b, p]:
                    assert t == end
                    at = sc[b, p]
                else:
                    assert not 96 <= t < 128
                    at = sc[b, p] + logp[b * W + p, t]
                assert abs(at - host(new)[b, n]) <= tol_log(at) and (p, t) not in taken
                taken.add((p, t))
        hist = lp.lp_beam_reorder(hist, parents)
        hist[:, k] = tokens.view(-1)
        used = lp.lp_beam_reorder(cache[:, :, :, :k], parents, dim=1)
        cache = torch.full_like(cache, 5.0)
        cache[:, :, :, :k] = used
        finished = finished.gather(1, parents.long()) | (tokens == end)
        scores = new
        rows = (pa + np.arange(B)[:, None] * W).reshape(-1)
        ref_hist = ref_hist[rows]
        ref_hist[:, k] = to.reshape(-1)
        ref_cache = ref_cache[:, rows]
        assert np.array_equal(host(hist)[:, :k + 1], ref_hist[:, :k + 1])
        assert np.array_equal(host(cache[:, :, :, :k].float()), ref_cache[:, :, :, :k])
    assert bool((scores <= 0).all())


def _steps(seed, dtype="bf16"):
    """Inputs of every call, and a function that makes the calls on them."""
    torch, lp = _torch(), _lp()
    rng = np.random.default_rng(seed)
    T, h, V, K, B, W = 40, 400, 9001, 20, 5, 8
    q, s = _fp8_head(np.random.default_rng(1), V, h)
    x = torch.from_numpy(rng.normal(0, 1, (T, h))).cuda().bfloat16()
    student = to_dev_bits(peaked(rng, T, V, dtype)[0], dtype)
    mask = torch.from_numpy(rng.random(T) < 0.8).cuda()
    g = torch.from_numpy(rng.normal(0, 1, T).astype(np.float32)).cuda()
    scores = torch.from_numpy(-rng.uniform(0, 9, (B, W)).astype(np.float32)).cuda()
    finished = torch.from_numpy(rng.random((B, W)) < 0.2).cuda()
    state = torch.from_numpy(rng.normal(0, 1, (2, B * W, 3, 50))).cuda().half()

    def step(stream=None):
        k = dict(stream=stream)
        few = lp.lp_lm_head_fp8_logits(x[:9], q, s, **k)
        more = lp.lp_lm_head_fp8_logits(x[:30], q, s, **k)
        t = lp.lp_lm_head_fp8_logits(x, q, s, out_dtype=torch.float32, **k)
        top = lp.lp_top_logits(t, K, mask, 1.2, **k)
        whole = lp.lp_top_logits(t[:1], K, None, 1.0, **k)
        f = lp.lp_distill_top(student, *top[:3], mask, 1.2, **k)
        d = lp.lp_distill_top_backward(student, *top[:3], mask, 1.2, f[1], f[2], g, **k)
        beams = lp.lp_beam_select(student, scores, 12, finished, 3, 0.8, **k)
        r = lp.lp_beam_reorder(state, beams[1], dim=1, **k)
        return [few, more, t, *top, *whole, *f, d, *beams, r]

    return [x, student, mask, g, scores, finished, state], step


def _equal(p, q):
    torch = _torch()
    return all(torch.equal(a.view(torch.uint8) if a.dim() else a, b.view(torch.uint8) if b.dim() else b)
               for a, b in zip([a.contiguous() for a in p], [b.contiguous() for b in q]))


def test_captured_and_replayed():
    """Two graphs of every call, replayed in turn with other inputs and eager calls between: the same bits as eager calls."""
    torch = _torch()
    inputs, step = _steps(2)
    others = [_steps(20 + k)[0] for k in range(3)]
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
            eager_again = step()  # behind the replay
            torch.cuda.synchronize()
            assert _equal(got[n], eager), (k, n)
            assert _equal(eager_again, eager), (k, n)
    # at once, on two streams
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for graph, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    assert _equal(got[0], eager) and _equal(got[1], eager)


def test_two_streams_at_once_and_inputs_unchanged():
    torch = _torch()
    both = [_steps(4), _steps(5)]
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
    """A workspace is scratch: what an earlier call of another kind or size left in it changes nothing."""
    torch, lp = _torch(), _lp()
    inputs, _ = _steps(6)
    x, student, _, _, scores, finished, _ = inputs
    q, s = _fp8_head(np.random.default_rng(1), 9001, 400)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    ids, logp = torch.arange(28, device="cuda").view(4, 7) * 11, torch.full((4, 7), -2.0, device="cuda")
    calls = (lambda w: [lp.lp_lm_head_fp8_logits(x, q, s, workspace=w)],
             lambda w: lp.lp_top_logits(student[:3], 7, None, 1.0, workspace=w),
             lambda w: lp.lp_beam_select(student, scores, 12, finished, 3, 0.8, workspace=w),
             lambda w: lp.lp_distill_top(student[:4], ids, logp, None, None, 1.0, workspace=w))
    for call in calls:
        want = call(None)
        for fill in (0, 255, 0x7f):
            ws.fill_(fill)
            assert _equal(call(ws), want)


def test_no_requests():
    """A batch that has run empty."""
    torch, lp = _torch(), _lp()
    scores, parents, tokens = lp.lp_beam_select(torch.zeros(0, 100, device="cuda"), torch.zeros(0, 4, device="cuda"))
    assert scores.shape == parents.shape == tokens.shape == (0, 4)
    state = torch.zeros(2, 0, 8, 3, device="cuda")
    assert lp.lp_beam_reorder(state, parents, dim=1).shape == state.shape
    assert lp.lp_beam_reorder(torch.zeros(3, 8, 0, device="cuda"), torch.zeros(2, 4, dtype=torch.int32, device="cuda"),
                              dim=1).shape == (3, 8, 0)
    ids, logp, rest, lse = lp.lp_top_logits(torch.zeros(0, 100, device="cuda"), 5)
    loss, lse, lse_rest = lp.lp_distill_top(torch.zeros(0, 100, device="cuda"), ids, logp, rest)
    g = lp.lp_distill_top_backward(torch.zeros(0, 100, device="cuda"), ids, logp, rest, None, 1.0, lse, lse_rest, loss)
    assert g.shape == (0, 100)


@pytest.mark.parametrize("tau", [1e-4, 0.02, 30.0, 1e6])
@pytest.mark.parametrize("V", [900, 12007])
def test_temperatures_far_from_one(tau, V):
    """Rows as good as one-hot, and as good as flat."""
    torch, lp = _torch(), _lp()
    rng = np.random.default_rng(3)
    bits, z = peaked(rng, 6, V, "fp32")
    x = to_dev(bits)
    K = 11
    got = [host(t) for t in lp.lp_top_logits(x, K, None, tau)]
    want = O.top_logits(z, K, None, tau)
    assert np.array_equal(got[0], want[0])
    # z / tau is taken with 1 / tau in fp64, exponents with log2(e) / tau in fp32: off by 2^-24 of themselves
    far = 2.0 ** -23 * np.abs(z).max() / tau
    for g, w in zip(got[1:], want[1:]):
        close(g, w, tol_log(w, 2) + np.where(np.abs(w) < 80, 0, far))
    ids, logp, rest = got[0], np.maximum(got[1], -60.0).astype(np.float32), np.maximum(got[2], -60.0).astype(np.float32)
    y = to_dev((bits + rng.normal(0, 1, bits.shape) * min(tau, 1.0)).astype(np.float32))
    z = host(y.double())
    a = [to_dev(t) for t in (ids, logp, rest)]
    loss, lse, lse_rest = lp.lp_distill_top(y, *a, None, tau)
    l_o, lse_o, lr_o = O.distill_top(z, ids, logp, rest, None, tau)
    close(host(lse), lse_o, tol_log(lse_o))
    close(host(lse_rest), lr_o, tol_log(lr_o))
    # terms of some (z / tau) each, in fp64, with masses off by 2^-23
    close(host(loss), l_o, 4 * SUM + 2.0 ** -22 * (np.abs(l_o) + 1))
    s = torch.zeros(2, 3, device="cuda")
    sc, pa, to = [host(t) for t in lp.lp_beam_select(x, s, 5, None, 0, tau)]
    sc_o, pa_o, to_o = O.beam_select(host(x.double()), np.zeros((2, 3), dtype=np.float32), 5, None, 0, tau)
    close(sc, sc_o, tol_log(sc_o, 2))


@pytest.mark.parametrize("T", [8, 20, 50, 100, 300])
def test_an_8_bit_head_past_four_gigabytes(T):
    torch, lp = _torch(), _lp()
    V, h = 600064, 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.empty(V, h, dtype=torch.uint8, device="cuda")
    q[:1000].random_(0, 64, generator=g)
    for v in range(1000, V, 100000):  # rows that repeat: cheap to fill
        n = min(100000, V - v)
        q[v:v + n] = q[:1000].repeat(100, 1)[:n]
    q[-256:].random_(64, 120, generator=g)
    q = q.view(torch.float8_e4m3fn)
    s = torch.rand(V // 128, h // 128, device="cuda", generator=g) + 0.5
    x = torch.randn(T, h, device="cuda", generator=g).bfloat16()
    whole = lp.lp_lm_head_fp8_logits(x, q, s)
    assert torch.equal(whole[:, -256:], lp.lp_lm_head_fp8_logits(x, q[-256:], s[-2:]))
    assert torch.equal(whole[:, 300032:300288], lp.lp_lm_head_fp8_logits(x, q[300032:300288], s[2344:2346]))
