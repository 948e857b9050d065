"""GPU parity of the 4-bit head against the fp64 oracle.

Quantiser: whole numbers and scales are equal.  Logits: terms are at most
(31 + 24) |x| s in magnitude (a nibble is used as 16 + q and the sum shifted
by 24); each is added through at most 32 (inside one matrix instruction) + 8
(start value and steps of a group) + ceil(h / 512) + 4 (groups of a wave, waves)
fp32 additions of relative error 2^-24, then rounded once to the type."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.helpers import host, to_dev, to_dev_bits
from tests.rules_cases import EPS, to_bits

pytestmark = pytest.mark.gpu
OUT = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def _torch():
    import torch
    return torch


def _dev(bits, dtype):
    return to_dev(bits) if dtype == "fp32" else to_dev_bits(bits, dtype)


def _pack(q):
    return (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)


def _head(V, h, group, seed):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 16, (V, h))
    s = to_bits(rng.uniform(0.002, 0.02, (V, -(-h // group))), "bf16")
    return q, s


def _tol(x, s, group, want, out):
    h = x.shape[1]
    mag = np.abs(x) @ np.repeat(s, group, axis=1)[:, :h].T * 55
    return (32 + 8 + -(-h // 512) + 4) * 2.0 ** -24 * mag + EPS[out] / 2 * np.abs(want) + 2.0 ** -25


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V,h,group", [(1, 32, 32), (3, 32, 128), (7, 96, 64), (33, 160, 128), (5, 4096, 32), (64, 1312, 64)])
def test_quantize(dtype, V, h, group):
    torch = _torch()
    rng = np.random.default_rng(V * h)
    w = rng.normal(0, 0.05, (V, h + 8))
    w[0, :40] = 0  # a group of zeros at the smallest sizes
    if V > 2:
        w[1] *= 1e-30 if dtype != "fp16" else 1e-3
        w[2] *= 1e30 if dtype != "fp16" else 1e3
    bits = to_bits(w, dtype)
    x = _dev(bits, dtype)
    for off in (0, 3):  # rows on and off the 16-byte grid
        q_o, s_o = O.w4_quantize(O.widen(bits, dtype)[:, off:off + h].astype(np.float32), group)
        p, s = _lp().lp_lm_head_w4_quantize(x[:, off:off + h], group)
        assert np.array_equal(host(p), _pack(q_o)) and np.array_equal(host(s.float()), s_o)
    pitch = torch.zeros((V, (h // 2 + 31) // 16 * 16), dtype=torch.uint8, device="cuda")
    sp = torch.zeros((V, 200), dtype=torch.bfloat16, device="cuda")
    _lp().lp_lm_head_w4_quantize(x[:, 3:3 + h], group, packed=pitch[:, :h // 2], scales=sp[:, :s.shape[1]])
    assert torch.equal(pitch[:, :h // 2], p) and not pitch[:, h // 2:].any()
    assert torch.equal(sp[:, :s.shape[1]], s) and not sp[:, s.shape[1]:].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,h,V,group", [
    (1, 32, 1, 32), (1, 32, 5, 128), (1, 64, 17, 64), (2, 96, 31, 32), (3, 160, 33, 128), (15, 224, 70, 64), (16, 512, 65, 128),
    (17, 544, 64, 32), (33, 1120, 130, 64), (48, 96, 47, 128), (49, 2080, 95, 32), (64, 128, 200, 128), (65, 192, 129, 64),
    (200, 352, 41, 32), (1, 5120, 300, 128), (40, 7168, 100, 32)])
def test_logits(dtype, out, T, h, V, group):
    torch = _torch()
    q, s = _head(V, h, group, T + h + V)
    xb = to_bits(np.random.default_rng(T).normal(0, 1, (T, h + 8)), dtype)
    x = O.widen(xb, dtype)[:, 8:]
    s64 = O.widen(s, "bf16")
    want = O.w4_logits(x, q, s64, group)
    tol = _tol(x, s64, group, want, out)
    hid, p, sc = to_dev_bits(xb, dtype)[:, 8:], to_dev(_pack(q)), to_dev_bits(s, "bf16")
    if h % 8 == 0 and (h + 8) % 8 == 0:
        got = host(_lp().lp_lm_head_w4_logits(hid, p, sc, group, out_dtype=getattr(torch, OUT[out])).float())
        assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) / tol).max())
    # pitches wider than the rows, and an output off the 16-byte grid
    buf = torch.full((T, V + 5), 7.0, dtype=getattr(torch, OUT[out]), device="cuda")
    pp = torch.full((V, h // 2 + 16), 255, dtype=torch.uint8, device="cuda")
    pp[:, :h // 2] = p
    ss = torch.full((V, sc.shape[1] + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    ss[:, 1:-2] = sc
    _lp().lp_lm_head_w4_logits(hid, pp[:, :h // 2], ss[:, 1:-2], group, out=buf[:, 2:2 + V])
    b = host(buf.float())
    assert np.array_equal(b[:, 2:2 + V], got) and np.all(b[:, :2] == 7) and np.all(b[:, 2 + V:] == 7)


def test_rows_do_not_depend_on_each_other():
    """Each of 70 rows alone gives the bits it has among the others, a row of
    NaN beside it included."""
    torch = _torch()
    q, s = _head(129, 1184, 64, 5)
    x = torch.randn(70, 1184, device="cuda").bfloat16()
    x[3] = float("nan")
    p, sc = to_dev(_pack(q)), to_dev_bits(s, "bf16")
    f = lambda a: _lp().lp_lm_head_w4_logits(a, p, sc, 64, out_dtype=torch.float32)  # noqa: E731
    whole = f(x)
    assert torch.isnan(whole[3]).all() and torch.isfinite(whole[torch.arange(70) != 3]).all()
    for n in (1, 16, 33, 64):
        part = f(x[:n])
        assert torch.equal(part.view(torch.int32), whole[:n].view(torch.int32)) or n > 3 and torch.equal(
            torch.nan_to_num(part), torch.nan_to_num(whole[:n]))
    for t in (0, 17, 69):
        assert torch.equal(f(x[t:t + 1])[0], whole[t])


def test_scale_nan_stays_in_its_row():
    torch = _torch()
    w = torch.randn(40, 256, device="cuda")
    w[7, 130], w[9, 3] = float("nan"), float("inf")
    p, s = _lp().lp_lm_head_w4_quantize(w, 128)
    out = _lp().lp_lm_head_w4_logits(torch.randn(2, 256, device="cuda").half(), p, s, 128)
    bad = torch.isnan(out).all(0)
    assert bad[7] and bad[9] and int(bad.sum()) == 2 and torch.isfinite(out[:, ~bad]).all()


def test_quantized_head_is_near_the_dense_one():
    """Each weight is off by at most half a step, amax / 7 / 2 (1 + 2^-8), and
    by half a step more where the rounded scale clips the largest."""
    torch = _torch()
    w = torch.randn(100, 384, device="cuda").bfloat16()
    p, s = _lp().lp_lm_head_w4_quantize(w, 64)
    eye = torch.eye(384, device="cuda").bfloat16()
    back = _lp().lp_lm_head_w4_logits(eye, p, s, 64, out_dtype=torch.float32).t()
    step = s.float().repeat_interleave(64, 1)
    assert bool(((back - w.float()).abs() <= step * (0.5 + 7 * 2.0 ** -8)).all())


def test_empty_and_offsets_past_32_bits():
    torch = _torch()
    lp = _lp()
    q, s = _head(40, 64, 32, 1)
    p, sc = to_dev(_pack(q)), to_dev_bits(s, "bf16")
    assert lp.lp_lm_head_w4_logits(torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda"), p, sc, 32).shape == (0, 40)
    V, h = 600000, 16384  # 4.9 GB packed
    x = torch.randn(2, h, device="cuda").half()
    big = torch.full((V, h // 2), 0x88, dtype=torch.uint8, device="cuda")
    scb = torch.full((V, h // 128), 0.01, dtype=torch.bfloat16, device="cuda")
    q, s = _head(3, h, 128, 2)
    big[-3:] = to_dev(_pack(q))
    scb[-3:] = to_dev_bits(s, "bf16")
    out = lp.lp_lm_head_w4_logits(x, big, scb, 128, out_dtype=torch.float32)
    alone = lp.lp_lm_head_w4_logits(x, big[-3:].clone(), scb[-3:].clone(), 128, out_dtype=torch.float32)
    assert torch.equal(out[:, -3:], alone) and float(out[:, :-3].abs().max()) < 1e-3
    w = torch.zeros((V, 8192), dtype=torch.bfloat16, device="cuda")  # 9.8 GB dense
    w[-1] = torch.randn(8192, device="cuda")
    p, s = lp.lp_lm_head_w4_quantize(w, 64)
    p1, s1 = lp.lp_lm_head_w4_quantize(w[-1:].clone(), 64)
    assert torch.equal(p[-1], p1[0]) and torch.equal(s[-1], s1[0]) and bool((p[:-1] == 0x88).all()) and not s[:-1].any()


def test_decode_step_captured_and_on_another_stream():
    """One step of a serving loop: the token's embedding, the 4-bit head, the
    rules in place, and the score of the drawn token; captured, replayed on
    new tokens, against the eager calls and the fp64 oracle."""
    torch = _torch()
    lp = _lp()
    rng = np.random.default_rng(4)
    B, h, V, L = 6, 256, 3001, 30
    Wb = to_bits(rng.normal(0, 0.3, (V, h)), "bf16")
    W = to_dev_bits(Wb, "bf16")
    p, s = lp.lp_lm_head_w4_quantize(W, 64)
    q_o, s_o = O.w4_quantize(O.widen(Wb, "bf16").astype(np.float32), 64)
    tok = to_dev(rng.integers(0, V, B).astype(np.int64))
    drawn = to_dev(rng.integers(0, V, B).astype(np.int64))
    buf = to_dev(rng.integers(0, V, (B, L)).astype(np.int32))
    lens = to_dev(np.full(B, 9, dtype=np.int32))
    pen = torch.full((B,), 0.4, device="cuda")
    words = torch.full((B, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    words[:, 5] = 0
    rules = lp.LogitRules(tokens=buf, hist_len=lens, presence=pen, frequency=pen, allowed=words)

    def step(stream=None):
        x = lp.lp_embedding(W, tok, 2.0, stream=stream)
        z = lp.lp_lm_head_w4_logits(x, p, s, 64, out_dtype=torch.float32, stream=stream)
        score = lp.lp_processed_logprobs_entropy(z, rules, drawn, None, 0.8, stream=stream)
        lp.lp_process_logits(z, rules, out=z, stream=stream)
        again = lp.lp_logprobs_entropy(z, drawn, None, 0.8, stream=stream)
        return [x, z, *score, *again]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    side = torch.cuda.Stream()
    for k in range(4):
        tok.copy_(to_dev(rng.integers(0, V, B).astype(np.int64)))
        d = rng.integers(0, V, B)
        drawn.copy_(to_dev(np.where((d // 32) == 5, 0, d).astype(np.int64)))
        buf[:, 9 + k] = tok.int()
        lens += 1
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), k
        other = step(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(other, eager)), k
        x64 = O.widen(host(got[0].view(torch.int16)).view(np.uint16), "bf16")
        n = int(lens[0])
        allowed = np.ones((B, V), dtype=bool)
        allowed[:, 160:192] = False
        z, _ = O.apply_rules(O.w4_logits(x64, q_o, s_o, 64), None, host(buf)[:, :n], None, host(pen), host(pen), None, allowed)
        lp_o, H_o, _ = O.logprobs_entropy(z, host(drawn), None, 0.8)
        # the logits' own error (see the head of this file) carries into the scores
        e = float(_tol(x64, s_o.astype(np.float64), 64, np.zeros_like(z), "fp32").max()) / 0.8
        for a, b, t in ((got[2], lp_o, 2 * e + 1e-5), (got[3], H_o, 40 * e + 1e-5), (got[5], lp_o, 2 * e + 1e-5)):
            assert np.abs(host(a) - b).max() <= t


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 16, 17, 33, 49, 64])
def test_the_same_bits_on_every_call(T, group):
    """And no NaN, which a register read before it is written would bring now
    and then."""
    torch = _torch()
    for h, V in ((1120, 700), (2048, 700), (5120, 90)):
        q, s = _head(V, h, group, h)
        x, p, sc = torch.randn(T, h, device="cuda").bfloat16(), to_dev(_pack(q)), to_dev_bits(s, "bf16")
        first = _lp().lp_lm_head_w4_logits(x, p, sc, group, out_dtype=torch.float32)
        assert torch.isfinite(first).all()
        for _ in range(8):
            assert torch.equal(_lp().lp_lm_head_w4_logits(x, p, sc, group, out_dtype=torch.float32), first)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,h,V,group", [(64, 512, 300, 32), (70, 768, 515, 64), (129, 2304, 257, 128)])
def test_blocks_of_64_rows_of_whole_chunk_pairs(dtype, T, h, V, group):
    """Several ranges of chunks and no column past the last pair."""
    q, s = _head(V, h, group, T + h)
    xb = to_bits(np.random.default_rng(T).normal(0, 1, (T, h)), dtype)
    x, s64 = O.widen(xb, dtype), O.widen(s, "bf16")
    want = O.w4_logits(x, q, s64, group)
    f = lambda a: host(_lp().lp_lm_head_w4_logits(a, to_dev(_pack(q)), to_dev_bits(s, "bf16"), group,  # noqa: E731
                                                  out_dtype=_torch().float32))
    hid = to_dev_bits(xb, dtype)
    got = f(hid)
    assert np.all(np.abs(got - want) <= _tol(x, s64, group, want, "fp32"))
    assert np.array_equal(f(hid[:40]), got[:40]) and np.array_equal(f(hid[3:8]), got[3:8])
