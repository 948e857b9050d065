"""CPU checks of the 4-bit head: every refusal of the binding and of the C entry points."""
import numpy as np
import pytest
import torch

import entropy_chunked_row_amd as lp
from oracle import lp_oracle as O

FAKE = 0x10000  # never dereferenced


def test_oracle_worked_group():
    w = np.zeros((1, 32), dtype=np.float32)
    w[0, :4] = [7.0, -3.5, 0.5, 1.5]  # scale 1: ties go to even
    q, s = O.w4_quantize(w, 32)
    assert s.tolist() == [[1.0]] and q[0, :5].tolist() == [15, 4, 8, 10, 8]
    assert O.w4_logits(np.ones((1, 32)), q, s, 32).tolist() == [[7.0 - 4 + 0 + 2]]


def test_binding_refusals():
    w, x = torch.zeros(10, 64), torch.zeros(3, 64, dtype=torch.bfloat16)
    p, s = torch.zeros(10, 32, dtype=torch.uint8), torch.zeros(10, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="group"):
        lp.lp_lm_head_w4_quantize(w, 48)
    with pytest.raises(ValueError, match="packed must"):
        lp.lp_lm_head_w4_quantize(w, 32, packed=torch.zeros(10, 31, dtype=torch.uint8))
    with pytest.raises(ValueError, match="scales must"):
        lp.lp_lm_head_w4_quantize(w, 32, scales=torch.zeros(10, 2))
    with pytest.raises(TypeError):
        lp.lp_lm_head_w4_quantize(w.double(), 32)
    with pytest.raises(ValueError, match="device"):
        lp.lp_lm_head_w4_quantize(w, 32)
    with pytest.raises(TypeError, match="uint8"):
        lp.lp_lm_head_w4_logits(x, p.int(), s, 32)
    with pytest.raises(TypeError, match="bfloat16"):
        lp.lp_lm_head_w4_logits(x, p, s.float(), 32)
    with pytest.raises(ValueError, match="disagree"):
        lp.lp_lm_head_w4_logits(x, p, s, 64)
    with pytest.raises(ValueError, match="disagree"):
        lp.lp_lm_head_w4_logits(x[:, :32], p, s, 32)
    with pytest.raises(ValueError, match="group"):
        lp.lp_lm_head_w4_logits(x, p, s, 16)
    with pytest.raises(ValueError, match="out must"):
        lp.lp_lm_head_w4_logits(x, p, s, 32, out=torch.zeros(3, 11))
    with pytest.raises(ValueError, match="out must"):
        lp.lp_lm_head_w4_logits(x, p, s, 32, out=torch.zeros(3, 10), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        lp.lp_lm_head_w4_logits(x, p, s, 32)


@pytest.mark.parametrize("over,code", [
    (dict(V=0), 1), (dict(V=2**31), 1), (dict(h=0), 1), (dict(h=48), 2), (dict(group=16), 2), (dict(group=256), 2),
    (dict(ldp=31), 1), (dict(ldp=40), 2), (dict(lds=1), 1), (dict(packed=None), 1), (dict(packed=FAKE + 8), 2),
    (dict(scales=None), 1), (dict(scales=FAKE + 1), 1), (dict(ldp=2**60), 2), (dict(lds=2**60), 2)])
def test_c_refusals_of_the_head(lib_handle, over, code):
    d = dict(V=10, h=64, group=32, packed=FAKE, ldp=32, scales=FAKE, lds=2)
    d.update(over)
    L = lib_handle
    assert L.lp_lm_head_w4_quantize(FAKE, 0, d["V"], d["h"], 2**20, d["group"], d["packed"], d["ldp"], d["scales"], d["lds"],
                                    None) == code
    assert L.lp_lm_head_w4_logits(FAKE, 0, 3, d["h"], 2**20, d["packed"], d["ldp"], d["scales"], d["lds"], d["V"], d["group"],
                                  FAKE, 0, 2**32, None) == code
    assert L.lp_last_error() != b""


@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), 2), (dict(dtype=7), 1), (dict(od=7), 1), (dict(T=-1), 1), (dict(ldh=56), 1), (dict(ldh=68), 2),
    (dict(ldo=9), 1), (dict(x=None), 1), (dict(x=FAKE + 8), 2), (dict(out=None), 1), (dict(out=FAKE + 1), 1),
    (dict(T=2**41), 2), (dict(T=0, x=None, out=None), 0)])
def test_c_refusals_of_the_logits(lib_handle, over, code):
    d = dict(x=FAKE, dtype=0, T=3, ldh=64, out=FAKE, od=2, ldo=10)
    d.update(over)
    assert lib_handle.lp_lm_head_w4_logits(d["x"], d["dtype"], d["T"], 64, d["ldh"], FAKE, 32, FAKE, 2, 10, 32, d["out"], d["od"],
                                           d["ldo"], None) == code


def test_c_refusals_of_the_quantizer(lib_handle):
    f = lib_handle.lp_lm_head_w4_quantize
    assert f(FAKE, 9, 10, 64, 64, 32, FAKE, 32, FAKE, 2, None) == 1
    assert f(FAKE, 0, 10, 64, 63, 32, FAKE, 32, FAKE, 2, None) == 1
    assert f(None, 0, 10, 64, 64, 32, FAKE, 32, FAKE, 2, None) == 1
    assert f(FAKE + 1, 0, 10, 64, 64, 32, FAKE, 32, FAKE, 2, None) == 1
    assert f(FAKE, 0, 10, 64, 2**60, 32, FAKE, 32, FAKE, 2, None) == 2
