"""CPU checks of the calls under logit rules: the oracle's formulas against
hand-worked rows and differences, and every refusal of the binding and of the
C entry points (all of which return before anything is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import entropy_chunked_row_amd as lp
from entropy_chunked_row_amd import _lib
from oracle import lp_oracle as O
from tests.rules_cases import Rules

FAKE = 0x10000  # never dereferenced


# ---------------------------------------------------------------------------
# oracle
# ---------------------------------------------------------------------------

def test_oracle_worked_row():
    z, slope = O.apply_rules([[2.0, -2.0, 1.0, 0.0, 5.0]], prompts=[[0, 9, -1]], outputs=[[1, 1, 2]], repetition=[2.0],
                             frequency=[0.25], presence=[0.5], biases=[[(3, 9.0), (3, 1.5), (7, 1.0)]],
                             allowed=np.array([[True, True, True, True, False]]))
    assert z.tolist() == [[1.0, -4.0 - 0.5 - 0.5, 0.5 - 0.25 - 0.5, 1.5, -np.inf]]
    assert slope.tolist() == [[0.5, 2.0, 0.5, 1.0, 0.0]]


def test_oracle_gradient_against_differences():
    c = Rules(6, 23, "fp32", seed=4, empty_row=False)
    x = c.logits64()
    g, gh = np.linspace(-1, 1, 6), np.linspace(0.4, -0.2, 6)
    tau = 0.8

    def loss(a):
        z, _ = O.apply_rules(a, **c.oracle)
        lpv, H, _ = O.logprobs_entropy(z, c.targets, c.mask, tau)
        return float((g * lpv + gh * H)[c.mask != 0].sum())

    z, slope = O.apply_rules(x, **c.oracle)
    d = O.processed_backward(z, slope, c.targets, c.mask, tau, g, gh)
    h = 1e-6
    for t in range(6):
        for j in range(23):
            up, dn = x.copy(), x.copy()
            up[t, j] += h
            dn[t, j] -= h
            assert abs((loss(up) - loss(dn)) / (2 * h) - d[t, j]) < 1e-7, (t, j)


# ---------------------------------------------------------------------------
# binding
# ---------------------------------------------------------------------------

T, V = 6, 100


def _parts(**over):
    d = dict(tokens=torch.zeros(T, 9, dtype=torch.int32), hist_len=torch.zeros(T, dtype=torch.int32),
             prompt_len=torch.zeros(T, dtype=torch.int32), repetition=torch.ones(T), frequency=torch.ones(T),
             presence=torch.ones(T), bias_offsets=torch.zeros(T + 1, dtype=torch.int64),
             bias_tokens=torch.zeros(3, dtype=torch.int32), bias_values=torch.zeros(3),
             allowed=torch.zeros(T, 4, dtype=torch.int32))
    d.update(over)
    return d


@pytest.mark.parametrize("over,err", [
    (dict(tokens=torch.zeros(T, 9, dtype=torch.int64)), TypeError),
    (dict(tokens=torch.zeros(T, 18, dtype=torch.int32)[:, ::2]), ValueError),
    (dict(tokens=None), ValueError),
    (dict(hist_len=None), ValueError),
    (dict(hist_len=torch.zeros(T, dtype=torch.int64)), TypeError),
    (dict(repetition=torch.ones(T, dtype=torch.float64)), TypeError),
    (dict(presence=torch.ones(2 * T)[::2]), ValueError),
    (dict(bias_offsets=torch.zeros(T + 1, dtype=torch.int32)), TypeError),
    (dict(bias_offsets=None), ValueError),
    (dict(bias_tokens=None), ValueError),
    (dict(bias_values=torch.zeros(2)), ValueError),
    (dict(allowed=torch.zeros(T, 4, dtype=torch.int64)), TypeError),
    (dict(allowed=torch.zeros(T, 4, dtype=torch.bool)), TypeError),
])
def test_rules_refuse_wrong_types_and_layouts(over, err):
    with pytest.raises(err):
        lp.LogitRules(**_parts(**over))


@pytest.mark.parametrize("over,match", [
    (dict(hist_len=torch.zeros(T - 1, dtype=torch.int32)), "hist_len"),
    (dict(prompt_len=torch.zeros(T + 1, dtype=torch.int32)), "prompt_len"),
    (dict(row_seq=torch.zeros(T + 1, dtype=torch.int32)), "row_seq"),
    (dict(frequency=torch.zeros(1)), "frequency"),
    (dict(tokens=torch.zeros(T - 1, 9, dtype=torch.int32)), "tokens"),
    (dict(bias_offsets=torch.zeros(T, dtype=torch.int64)), "bias_offsets"),
    (dict(allowed=torch.zeros(T, 3, dtype=torch.int32)), "allowed"),
    (dict(allowed=torch.zeros(T - 1, 4, dtype=torch.int32)), "allowed"),
    (dict(), "device"),  # every length right: host tensors are refused next
])
def test_calls_refuse_wrong_lengths(over, match):
    r = lp.LogitRules(**_parts(**over))
    x, y, f = torch.zeros(T, V), torch.zeros(T, dtype=torch.int64), torch.zeros(T)
    for call in (lambda: lp.lp_process_logits(x, r), lambda: lp.lp_processed_logprobs_entropy(x, r, y),
                 lambda: lp.lp_processed_logprobs_entropy_backward(x, r, y, None, 1.0, f, f, f)):
        with pytest.raises(ValueError, match=match):
            call()


def test_calls_refuse_wrong_operands():
    x, y, f = torch.zeros(T, V), torch.zeros(T, dtype=torch.int64), torch.zeros(T)
    with pytest.raises(TypeError):
        lp.lp_process_logits(x.double(), None)
    with pytest.raises(ValueError, match="2-D"):
        lp.lp_process_logits(x[0], None)
    with pytest.raises(ValueError, match="contiguous rows"):
        lp.lp_process_logits(x.t(), None)
    with pytest.raises(ValueError, match="shape and dtype"):
        lp.lp_process_logits(x, None, out=x.bfloat16())
    with pytest.raises(ValueError, match="targets"):
        lp.lp_processed_logprobs_entropy(x, None, y[:-1])
    with pytest.raises(TypeError):
        lp.lp_processed_logprobs_entropy(x, None, y.int())
    with pytest.raises(ValueError, match="lse"):
        lp.lp_processed_logprobs_entropy_backward(x, None, y, None, 1.0, f[:-1], f, f)
    with pytest.raises(ValueError, match="grad_entropy"):
        lp.lp_processed_logprobs_entropy_backward(x, None, y, None, 1.0, f, f, f, f[:-1])


# ---------------------------------------------------------------------------
# C ABI
# ---------------------------------------------------------------------------

def _c_rules(**over):
    r = _lib.LogitRulesC()
    d = dict(tokens=FAKE, buffers=4, ld_tokens=8, max_len=8, hist_len=FAKE, repetition=FAKE, bias_offsets=FAKE,
             bias_tokens=FAKE, bias_values=FAKE, bias_count=5, allowed=FAKE, ld_allowed=1)
    d.update(over)
    for k, v in d.items():
        setattr(r, k, v)
    return ctypes.byref(r)


BAD_RULES = [dict(hist_len=None), dict(buffers=3), dict(buffers=0), dict(max_len=0), dict(ld_tokens=7),
             dict(max_len=2**31, ld_tokens=2**31), dict(buffers=2**31), dict(ld_tokens=2**40), dict(tokens=None),
             dict(tokens=FAKE + 2), dict(bias_offsets=FAKE + 4), dict(bias_tokens=None), dict(bias_offsets=None),
             dict(bias_count=-1), dict(bias_count=2**31), dict(ld_allowed=0), dict(allowed=FAKE + 1)]


@pytest.mark.parametrize("over", BAD_RULES, ids=lambda d: "-".join(f"{k}={v}" for k, v in d.items()))
def test_c_calls_refuse_bad_rules(lib_handle, over):
    L, r = lib_handle, _c_rules(**over)
    assert L.lp_process_logits(FAKE, 0, 4, 16, 16, r, None, 2 * FAKE, 16, None) == 1
    assert L.lp_processed_logprobs_entropy(FAKE, 0, 4, 16, 16, r, FAKE, None, 1.0, FAKE, None, None, FAKE, 1 << 20,
                                           None) == 1
    assert L.lp_processed_logprobs_entropy_backward(FAKE, 0, 4, 16, 16, r, FAKE, None, 1.0, FAKE, None, FAKE, None,
                                                    2 * FAKE, 16, None) == 1
    assert L.lp_last_error() != b""


@pytest.mark.parametrize("over,code", [
    (dict(dtype=9), 1), (dict(T=-1), 1), (dict(V=0), 1), (dict(V=2**31), 1), (dict(ld=15), 1), (dict(logits=None), 1),
    (dict(logits=FAKE + 1), 1), (dict(T=2**41), 2), (dict(ld=2**40), 2)])
def test_c_calls_refuse_bad_operands(lib_handle, over, code):
    L = lib_handle
    a = dict(logits=FAKE, dtype=0, T=4, V=16, ld=16)
    a.update(over)
    h = (a["logits"], a["dtype"], a["T"], a["V"], a["ld"])
    assert L.lp_process_logits(*h, None, None, 2 * FAKE, 2**31, None) == code
    assert L.lp_processed_logprobs_entropy(*h, None, FAKE, None, 1.0, FAKE, None, None, FAKE, 1 << 20, None) == code
    assert L.lp_processed_logprobs_entropy_backward(*h, None, FAKE, None, 1.0, FAKE, None, FAKE, None, 2 * FAKE, 2**31,
                                                    None) == code


def test_c_calls_refuse_the_rest(lib_handle):
    L = lib_handle
    h = (FAKE, 0, 4, 16, 16, None)
    # output: missing, narrow, misaligned, overlapping the input without being it
    for out, ld in ((None, 16), (2 * FAKE, 15), (2 * FAKE + 1, 16), (FAKE + 16, 16), (FAKE, 32), (FAKE - 32, 16)):
        assert L.lp_process_logits(*h, None, out, ld, None) == 1
    assert L.lp_process_logits(*h, None, 2 * FAKE, 2**40, None) == 2
    s = L.lp_processed_logprobs_entropy
    need = L.lp_processed_workspace_bytes(4, 16)
    assert need >= 4 * 16
    assert s(*h, None, None, 1.0, FAKE, None, None, FAKE, need, None) == 1
    assert s(*h, FAKE, None, 1.0, None, None, None, FAKE, need, None) == 1
    assert s(*h, FAKE + 4, None, 1.0, FAKE, None, None, FAKE, need, None) == 1
    assert s(*h, FAKE, None, float("nan"), FAKE, None, None, FAKE, need, None) == 1
    assert s(*h, FAKE, None, 1.0, FAKE, FAKE + 2, None, FAKE, need, None) == 1
    assert s(*h, FAKE, None, 1.0, FAKE, None, None, FAKE, need - 1, None) == 3
    assert s(*h, FAKE, None, 1.0, FAKE, None, None, None, need, None) == 3
    assert s(*h, FAKE, None, 1.0, FAKE, None, None, FAKE + 128, need, None) == 1
    b = L.lp_processed_logprobs_entropy_backward
    assert b(*h, None, None, 1.0, FAKE, None, FAKE, None, 2 * FAKE, 16, None) == 1
    assert b(*h, FAKE, None, 1.0, None, None, FAKE, None, 2 * FAKE, 16, None) == 1
    assert b(*h, FAKE, None, 1.0, FAKE, None, None, None, 2 * FAKE, 16, None) == 1
    assert b(*h, FAKE, None, 1.0, FAKE, None, FAKE, FAKE, 2 * FAKE, 16, None) == 1  # grad_entropy without entropy
    assert b(*h, FAKE, None, 1.0, FAKE, None, FAKE, None, None, 16, None) == 1
    assert b(*h, FAKE, None, 1.0, FAKE, None, FAKE, None, FAKE, 16, None) == 1  # the logits themselves
    assert b(*h, FAKE, None, float("inf"), FAKE, None, FAKE, None, 2 * FAKE, 16, None) == 1
    assert b(*h, FAKE, None, 1.0, FAKE, None, FAKE, None, 2 * FAKE, 15, None) == 1


def test_c_empty_calls_and_workspace(lib_handle):
    L = lib_handle
    assert L.lp_process_logits(None, 0, 0, 16, 16, None, None, None, 16, None) == 0
    assert L.lp_processed_logprobs_entropy(None, 0, 0, 16, 16, None, None, None, 1.0, None, None, None, None, 0, None) == 0
    assert L.lp_processed_logprobs_entropy_backward(None, 0, 0, 16, 16, None, None, None, 1.0, None, None, None, None,
                                                    None, 16, None) == 0
    f = L.lp_processed_workspace_bytes
    assert f(-1, 5) == 0 and f(4, 0) == 0 and f(4, 2**31) == 0 and f(0, 5) == 256
    for T_, V_ in ((1, 1), (1, 151936), (8192, 151936), (100000, 33)):
        assert f(T_, V_) % 256 == 0 and f(T_, V_) >= 16 * T_
