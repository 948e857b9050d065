"""GPU parity of the 8-bit head against the fp64 oracle.

Quantiser: values and scales are equal.  Logits: products of two e4m3 values are
exact; a block's 128 are added inside matrix instructions, each addition off by at
most 2^-23 of what has been added so far in magnitude (2^-24 where it rounds, twice
that where it cuts off; for 16-bit results the 8-bit instructions first drop, of each of 8 products, up to 2^-13
of the largest: 8 x 2^-13 of the magnitudes' sum at most); the block's sum is scaled by one rounded factor and added to
the others (3 roundings and one per block), at most 8 parts of them are joined, and
the result is rounded once to the type.  `mag` bounds every partial sum."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.choose_cases import close, dev_rows
from tests.helpers import host, to_dev, to_dev_bits
from tests.rules_cases import DTYPES, EPS, to_bits

pytestmark = pytest.mark.gpu
OUT = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def _torch():
    import torch
    return torch


def _head(V, h, seed):
    """(q float8 tensor on the device, scales, the same as fp64)."""
    torch = _torch()
    rng = np.random.default_rng(seed)
    w = np.clip(rng.normal(0, 110, (V, h)), -448, 448).astype(np.float32)
    q = torch.from_numpy(w).to(torch.float8_e4m3fn)
    s = rng.uniform(1e-4, 4e-4, (-(-V // 128), -(-h // 128))).astype(np.float32)
    return q.cuda(), to_dev(s), q.double().numpy(), s


def _tol(mag, h, want, out):
    blocks = -(-h // 128)
    return ((0 if out == "fp32" else 8 * 2.0 ** -13) + 128 * 2.0 ** -23 + (blocks + 3 + 8) * 2.0 ** -24) * mag + EPS[out] / 2 * np.abs(want) + (2.0 ** -25 if out == "fp16" else 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,h", [(1, 16), (3, 128), (127, 144), (129, 112), (300, 272), (128, 128), (260, 1040)])
def test_quantize(dtype, V, h):
    torch = _torch()
    rng = np.random.default_rng(V * h)
    w = rng.normal(0, 0.05, (V, h + 8))
    w[:, 3:40] *= 8
    if V > 130:
        w[128:] = 0                                             # a block of zeros
    if V > 260:
        w[256:] *= 0
        w[257, 5] = 1e-40 if dtype != "fp16" else 6e-8          # of tiny values
    bits = to_bits(w, dtype)
    x = dev_rows(bits, dtype)
    for off in (0, 3):  # rows on and off the 16-byte grid
        q_o, s_o = O.fp8_blocks(O.widen(bits, dtype)[:, off:off + h].astype(np.float32), 128)
        q, s = _lp().lp_lm_head_fp8_quantize(x[:, off:off + h])
        assert np.array_equal(host(s), s_o) and np.array_equal(host(q.float()), q_o)
    pitch = torch.zeros((V, (h + 31) // 16 * 16), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sp = torch.zeros((s.shape[0], s.shape[1] + 3), device="cuda")
    _lp().lp_lm_head_fp8_quantize(x[:, 3:3 + h], q=pitch[:, :h], scales=sp[:, :s.shape[1]])
    assert torch.equal(pitch[:, :h].float(), q.float()) and not pitch[:, h:].float().any()
    assert torch.equal(sp[:, :s.shape[1]], s) and not sp[:, s.shape[1]:].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_rounds_like_the_type(dtype):
    """Every bf16 magnitude between 2^-12 and 448 (what of it the type holds) beside a 448, so that the scale is 1 up to a
    rounding: ties, subnormals of the 8-bit type and both signs among them."""
    m = (np.arange(0x3980, 0x43e0, dtype=np.uint32) << 16).view(np.float32)
    n = -(-m.size * 2 // 127)
    w = np.zeros((n, 128), dtype=np.float32)
    w[:, 1:].flat[:m.size * 2] = np.concatenate([m, -m])
    w[:, 0] = 448
    bits = to_bits(w, dtype)
    q_o, s_o = O.fp8_blocks(O.widen(bits, dtype).astype(np.float32), 128)
    q, s = _lp().lp_lm_head_fp8_quantize(dev_rows(bits, dtype))
    assert np.array_equal(host(s), s_o) and np.array_equal(host(q.float()), q_o)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 3, 16, 17, 40, 64, 65, 130, 200, 300])
def test_hidden_rows_are_brought_to_8_bits(dtype, T):
    """Through a head that is the identity, with scales of 1: the logits are the rows' own values, to the last bit."""
    torch = _torch()
    h = 336
    q = torch.eye(h, device="cuda").to(torch.float8_e4m3fn)
    s = torch.ones(3, 3, device="cuda")
    xb = to_bits(np.random.default_rng(T).normal(0, 1, (T, h)) * np.exp2(np.random.default_rng(1).integers(-6, 6, (T, h))), dtype)
    xb[0, :128] = 0
    x_q, x_s = O.fp8_blocks(O.widen(xb, dtype).astype(np.float32), 1)
    want = (x_q * np.repeat(x_s.astype(np.float64), 128, 1)[:, :h]).astype(np.float32)
    got = host(_lp().lp_lm_head_fp8_logits(to_dev_bits(xb, dtype), q, s, out_dtype=torch.float32))
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype,out", [("bf16", "fp32"), ("fp16", "bf16"), ("bf16", "fp16"), ("fp16", "fp32"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,h,V", [
    (1, 16, 1), (1, 128, 5), (2, 144, 17), (7, 1040, 130), (8, 5120, 400), (16, 1024, 257), (16, 8192, 40), (9, 8208, 33),
    (17, 128, 255), (33, 272, 300), (64, 656, 513), (65, 128, 256), (100, 1296, 129), (128, 400, 1000), (129, 112, 257),
    (256, 384, 511), (257, 896, 300), (300, 2064, 700), (1000, 256, 260)])
def test_logits(dtype, out, T, h, V):
    torch = _torch()
    q, s, q64, s64 = _head(V, h, T + h + V)
    rng = np.random.default_rng(T)
    x = rng.normal(0, 1, (T, h + 3))
    x[:, rng.integers(0, h, 3)] *= 20
    xb = to_bits(x, dtype)
    want, mag = O.fp8_logits(O.widen(xb, dtype)[:, :h], q64, s64)
    tol = _tol(mag, h, want, out)
    hid = to_dev_bits(xb, dtype)[:, :h]  # rows off the 16-byte grid
    got = _lp().lp_lm_head_fp8_logits(hid, q, s, out_dtype=getattr(torch, OUT[out]))
    close(host(got.float()), want, tol)
    assert torch.equal(_lp().lp_lm_head_fp8_logits(hid.contiguous(), q, s, out_dtype=got.dtype), got)
    # pitches wider than the rows, NaN behind them, an output off the 16-byte grid
    buf = torch.full((T, V + 5), 7.0, dtype=got.dtype, device="cuda")
    qq = torch.full((V, h + 16), 0x7f, dtype=torch.uint8, device="cuda")
    qq[:, :h] = q.view(torch.uint8)
    ss = torch.full((s.shape[0], s.shape[1] + 2), float("nan"), device="cuda")
    ss[:, 1:-1] = s
    _lp().lp_lm_head_fp8_logits(hid, qq.view(torch.float8_e4m3fn)[:, :h], ss[:, 1:-1], out=buf[:, 2:2 + V])
    assert torch.equal(buf[:, 2:2 + V], got) and bool((buf[:, :2] == 7).all()) and bool((buf[:, 2 + V:] == 7).all())


@pytest.mark.parametrize("T", [5, 40, 100, 300])
def test_nan_and_infinity_stay_in_their_rows(T):
    torch = _torch()
    q, s, _, _ = _head(300, 400, 1)
    x = torch.randn(T, 400, device="cuda").bfloat16()
    clean = _lp().lp_lm_head_fp8_logits(x, q, s, out_dtype=torch.float32)
    x[1, 7], x[3, 399] = float("nan"), float("inf")
    got = _lp().lp_lm_head_fp8_logits(x, q, s, out_dtype=torch.float32)
    rows = torch.ones(T, dtype=torch.bool)
    rows[[1, 3]] = False
    assert torch.isnan(got[[1, 3]]).all() and torch.equal(got[rows], clean[rows])
    bad = q.clone().view(torch.uint8)
    bad[130, 5] = 0x7f
    got = _lp().lp_lm_head_fp8_logits(x[rows.cuda()], bad.view(torch.float8_e4m3fn), s, out_dtype=torch.float32)
    cols = torch.ones(300, dtype=torch.bool)
    cols[130] = False
    assert torch.isnan(got[:, 130]).all() and torch.equal(got[:, cols.cuda()], clean[rows.cuda()][:, cols.cuda()])


def test_empty():
    torch = _torch()
    q, s, _, _ = _head(30, 64, 1)
    assert _lp().lp_lm_head_fp8_logits(torch.zeros(0, 64, device="cuda").half(), q, s).shape == (0, 30)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("T,h,V", [
    (1, 16, 9001), (4, 1040, 12293), (16, 2064, 8209), (16, 7168, 5000), (16, 8192, 4113), (17, 16, 9001), (32, 1152, 12293),
    (31, 8192, 4200), (20, 5120, 5003), (33, 128, 40001), (40, 256, 33001), (64, 8208, 300), (65, 144, 33001), (128, 8320, 260),
    (300, 144, 20001)])
def test_logits_of_many_tiles(out, T, h, V):
    """Workgroups that walk over several tiles, K that leaves waves one block fewer or none, one to many blocks."""
    torch = _torch()
    q, s, q64, s64 = _head(V, h, T + h + V)
    rng = np.random.default_rng(V)
    xb = to_bits(rng.normal(0, 1, (T, h)), "bf16")
    want, mag = O.fp8_logits(O.widen(xb, "bf16"), q64, s64)
    hid = to_dev_bits(xb, "bf16")
    got = _lp().lp_lm_head_fp8_logits(hid, q, s, out_dtype=getattr(torch, OUT[out]))
    close(host(got.float()), want, _tol(mag, h, want, out))
    for _ in range(3):  # the same bits on every call
        assert torch.equal(_lp().lp_lm_head_fp8_logits(hid, q, s, out_dtype=got.dtype), got)
