"""CPU checks of the 8-bit head: the oracle's rounding against worked values and
torch's own type, and every refusal of the binding and of the C entry points."""
import numpy as np
import pytest
import torch

import entropy_chunked_row_amd as lp
from oracle import lp_oracle as O

FAKE = 0x10000  # never dereferenced


def test_oracle_rounding():
    assert O.e4m3([448, 449, 464, 17, 18, 19, 1.0625, 1.1875, 2.0**-9, 2.0**-10, 3 * 2.0**-10, 0, -0.3]).tolist() == [
        448, 448, 448, 16, 18, 20, 1.0, 1.25, 2.0**-9, 0, 2.0**-8, 0, -0.3125]
    assert np.isnan(O.e4m3([465.0, np.nan, -1e9])).all()
    x = np.random.default_rng(0).normal(0, 1, 20000).astype(np.float32) * np.float32(2.0) ** np.random.default_rng(1).integers(-12, 6, 20000)
    x = x[np.abs(x) <= 448]
    assert np.array_equal(O.e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_oracle_worked_block():
    x = np.zeros((2, 130), dtype=np.float32)
    x[0, 0], x[1, 3], x[0, 129] = 448.0, -1.0, 0.5
    q, s = O.fp8_blocks(x, 128)
    assert s.shape == (1, 2) and abs(s[0, 0] - 1) < 1e-6 and abs(s[0, 1] * 448 - 0.5) < 1e-6
    assert q[0, 0] == 448 and q[1, 3] == -1 and q[0, 129] == 448
    out, mag = O.fp8_logits(np.ones((1, 130)), q, s)
    assert np.allclose(out, [[448.5, -1.0]], rtol=1e-6) and np.allclose(mag, [[448.5, 1.0]], rtol=1e-6)
    assert O.fp8_scale(0.0) == np.float32(2.0**-126)


def test_binding_refusals():
    f8 = torch.float8_e4m3fn
    w, x = torch.zeros(300, 160), torch.zeros(3, 160, dtype=torch.bfloat16)
    q, s = torch.zeros(300, 160, dtype=torch.uint8).view(f8), torch.zeros(3, 2)
    with pytest.raises(TypeError):
        lp.lp_lm_head_fp8_quantize(w.double())
    with pytest.raises(ValueError, match="q must"):
        lp.lp_lm_head_fp8_quantize(w, q=q[:299])
    with pytest.raises(ValueError, match="q must"):
        lp.lp_lm_head_fp8_quantize(w, q=q.view(torch.uint8))
    with pytest.raises(ValueError, match="scales must"):
        lp.lp_lm_head_fp8_quantize(w, scales=torch.zeros(2, 2))
    with pytest.raises(ValueError, match="device"):
        lp.lp_lm_head_fp8_quantize(w)
    with pytest.raises(TypeError, match="float8"):
        lp.lp_lm_head_fp8_logits(x, q.view(torch.uint8), s)
    with pytest.raises(TypeError, match="float32"):
        lp.lp_lm_head_fp8_logits(x, q, s.half())
    with pytest.raises(ValueError, match="disagree"):
        lp.lp_lm_head_fp8_logits(x[:, :144], q, s)
    with pytest.raises(ValueError, match="disagree"):
        lp.lp_lm_head_fp8_logits(x, q, s[:2])
    with pytest.raises(ValueError, match="out must"):
        lp.lp_lm_head_fp8_logits(x, q, s, out=torch.zeros(3, 299))
    with pytest.raises(ValueError, match="out must"):
        lp.lp_lm_head_fp8_logits(x, q, s, out=torch.zeros(3, 300), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        lp.lp_lm_head_fp8_logits(x, q, s)


@pytest.mark.parametrize("over,code", [
    (dict(V=0), 1), (dict(V=2**31), 1), (dict(h=0), 1), (dict(h=24), 2), (dict(h=2**20 + 16, ldq=2**21), 2), (dict(ldq=144), 1),
    (dict(ldq=168), 2), (dict(ldq=2**23 + 16), 2), (dict(lds=1), 1), (dict(lds=2**60), 2), (dict(q=None), 1), (dict(q=0x20008), 2),
    (dict(s=None), 1), (dict(s=0x400002), 1)])
def test_c_refusals_of_the_head(lib_handle, over, code):
    d = dict(V=300, h=160, q=0x200000, ldq=160, s=0x400000, lds=2)
    d.update(over)
    L = lib_handle
    assert L.lp_lm_head_fp8_quantize(0x10000000, 0, d["V"], d["h"], 2**22, d["q"], d["ldq"], d["s"], d["lds"], None) == code
    assert L.lp_lm_head_fp8_logits(0x10000000, 0, 3, d["h"], 2**22, d["q"], d["ldq"], d["s"], d["lds"], d["V"], 0x20000000, 2,
                                   2**32, 0x500000, 1 << 30, None) == code
    assert L.lp_last_error() != b""


@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), 2), (dict(dtype=9), 1), (dict(od=9), 1), (dict(T=-1), 1), (dict(ldh=144), 1), (dict(ldo=299), 1),
    (dict(x=None), 1), (dict(x=FAKE + 1), 1), (dict(out=None), 1), (dict(out=0x800002), 1), (dict(T=2**37), 2), (dict(ws=None), 3),
    (dict(n=256), 3), (dict(ws=0x500080), 1), (dict(out=0x200000), 1), (dict(ws=0x200000), 1), (dict(out=FAKE), 1),
    (dict(out=0x400000), 1), (dict(ws=0x800000), 1), (dict(T=0, x=None, out=None, ws=None), 0)])
def test_c_refusals_of_the_logits(lib_handle, over, code):
    d = dict(x=FAKE, dtype=0, T=3, ldh=160, out=0x800000, od=2, ldo=300, ws=0x500000, n=1 << 20)
    d.update(over)
    assert lib_handle.lp_lm_head_fp8_logits(d["x"], d["dtype"], d["T"], 160, d["ldh"], 0x200000, 160, 0x400000, 2, 300, d["out"],
                                            d["od"], d["ldo"], d["ws"], d["n"], None) == code


def test_c_refusals_of_the_quantizer(lib_handle):
    f = lib_handle.lp_lm_head_fp8_quantize
    assert f(FAKE, 9, 300, 160, 160, 0x200000, 160, 0x400000, 2, None) == 1
    assert f(FAKE, 0, 300, 160, 159, 0x200000, 160, 0x400000, 2, None) == 1
    assert f(None, 0, 300, 160, 160, 0x200000, 160, 0x400000, 2, None) == 1
    assert f(FAKE + 1, 0, 300, 160, 160, 0x200000, 160, 0x400000, 2, None) == 1
    assert f(FAKE, 0, 300, 160, 2**60, 0x200000, 160, 0x400000, 2, None) == 2
    assert f(0x200000, 0, 300, 160, 160, 0x200000, 160, 0x400000, 2, None) == 1
    assert f(FAKE, 0, 300, 160, 160, 0x200000, 160, 0x200010, 2, None) == 1


def test_workspace_sizes(lib_handle):
    f = lib_handle.lp_lm_head_fp8_workspace_bytes
    # 2 blocks of a row and their scales (4 rows of them, 256 more behind), each up to 256 bytes
    assert f(1, 160, 300) == 256 + 1280 and f(0, 160, 300) == 1024
    for bad in ((-1, 160, 300), (1, 24, 300), (1, 0, 300), (1, 160, 0), (2**37, 160, 300), (1, 2**20 + 16, 300)):
        assert f(*bad) == 0
