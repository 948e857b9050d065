"""Entries of a teacher's list whose mass is nothing in fp32 (finite log-probs from finite masks), against students that
have no weight there: such an entry adds nothing to the loss, and a mass that is merely tiny still counts.

Tolerances are those of the other distillation tests (choose_cases): a log-sum is off by SUM, twice in a loss, times
the masses."""
import numpy as np
import pytest

from oracle import lp_oracle as O
from tests.choose_cases import SUM, close, dev_rows, grad_tol, lists, peaked, tol_log
from tests.helpers import host, to_dev
from tests.rules_cases import DTYPES, to_bits

pytestmark = pytest.mark.gpu
NONE = [-110.0, -800.0, -1e9, -3.4e38]


def _lp():
    import entropy_chunked_row_amd as lp
    return lp


def _rows(dtype, V, K):
    """Student rows (bits, fp64) and lists: 0 and 1 hold entries without mass where the student is -inf and where it is
    finite; 2 .. 5 a rest without mass while the student has none outside the list; 6 both; 7 and 8 an entry and a rest
    of e^-100, which is a mass, where the student has none; 9 an ordinary row."""
    rng = np.random.default_rng(V)
    bits, z = peaked(rng, 10, V, dtype)
    ids, lp, rest = lists(rng, z, K, 1.0, pad=False)
    z0 = z.copy()
    lp[[0, 1, 6], 2:6] = NONE
    for t in (0, 6):
        z0[t, ids[t, 2:6]] = -np.inf
    for t, r in zip((2, 3, 4, 5, 6), NONE + NONE[2:3]):
        rest[t] = r
        z0[t] = np.where(np.isin(np.arange(V), ids[t]), z0[t], -np.inf)
    lp[7, 3] = -100.0
    z0[7, ids[7, 3]] = -np.inf
    rest[8] = -100.0
    z0[8] = np.where(np.isin(np.arange(V), ids[8]), z0[8], -np.inf)
    bits = to_bits(z0, dtype)
    return bits, O.widen(bits, dtype), ids, lp, rest


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [900, 9001, 70001])
def test_entries_without_mass(dtype, V):
    import torch
    lp, K = _lp(), 12
    bits, z, ids, lpk, rest = _rows(dtype, V, K)
    x = dev_rows(bits, dtype)
    assert (lp.lp_distill_top_workspace_bytes({"bf16": 0, "fp16": 1, "fp32": 2}[dtype], 10, V) > 256) == (V == 70001)
    with np.errstate(invalid="ignore", over="ignore"):
        want = O.distill_top(z, ids, lpk, rest, None, 1.0)
    assert np.isfinite(want[0][[0, 1, 2, 3, 4, 5, 6, 9]]).all() and (want[0][[7, 8]] == np.inf).all()
    a = [to_dev(t) for t in (ids, lpk, rest)]
    got = lp.lp_distill_top(x, *a)
    mass = np.exp(lpk.astype(np.float64)).sum(1) + np.exp(rest.astype(np.float64))
    finite = np.where(np.isfinite(want[0]), np.abs(want[0]), 0)
    close(host(got[0]), want[0], 2 * SUM * (1 + mass) + 2.0 ** -24 * finite)
    for g, w in zip(got[1:], want[1:]):
        close(host(g), w, tol_log(w))
    g = np.linspace(0.5, 1.5, 10).astype(np.float32)
    d = lp.lp_distill_top_backward(x, *a, None, 1.0, got[1], got[2], to_dev(g))
    ref = O.distill_top_backward(z, ids, lpk, rest, None, 1.0, g)
    close(host(d.float()), ref, grad_tol(z, ids, lpk, rest, 1.0, g, ref, dtype))
    # rows in one slice and cut into several: the same rule (here many rows, so that each is one)
    if V == 70001:
        n = 100
        many = [t.repeat(n, *[1] * (t.dim() - 1)) for t in (x, *a)]
        assert lp.lp_distill_top_workspace_bytes({"bf16": 0, "fp16": 1, "fp32": 2}[dtype], 10 * n, V) == 256
        whole = lp.lp_distill_top(*many)[0]
        close(host(whole[-10:]), want[0], 2 * SUM * (1 + mass) + 2.0 ** -24 * finite)
        assert torch.equal(whole[:10], whole[-10:])


@pytest.mark.parametrize("V", [2000, 70001])
@pytest.mark.parametrize("low", [-1e4, -1e9, -3e38])
def test_a_teacher_under_finite_masks_and_a_student_under_rules(V, low):
    """A grammar leaves a few tokens: the teacher's logits hold a finite mask elsewhere, so its list runs on into masked
    tokens with finite log-probs; the student's hold -inf, from the rules.  What is left of the loss is the allowed part."""
    import torch
    lp = _lp()
    rng = np.random.default_rng(int(-low) % 97 + V)
    T, K = 6, 9
    allowed = np.zeros((T, V), dtype=bool)
    for t in range(T):
        allowed[t, rng.choice(V, 3 + t, replace=False)] = True
    words = np.zeros((T, -(-V // 32) * 32), dtype=np.uint8)
    words[:, :V] = allowed
    words = np.packbits(words, axis=1, bitorder="little").view(np.int32)
    teacher = to_dev(np.where(allowed, rng.normal(0, 2, (T, V)), low).astype(np.float32))
    student = lp.lp_process_logits(to_dev(rng.normal(0, 2, (T, V)).astype(np.float32)), lp.LogitRules(allowed=to_dev(words)))
    z = host(student).astype(np.float64)
    assert np.array_equal(np.isneginf(z), ~allowed)
    ids, logp, rest, _ = lp.lp_top_logits(teacher, K)
    t64 = host(teacher).astype(np.float64)
    ids_o, logp_o, rest_o, _ = O.top_logits(t64, K, None, 1.0)
    assert np.array_equal(host(ids), ids_o)
    close(host(logp), logp_o, tol_log(logp_o, 2))
    close(host(rest), rest_o, tol_log(rest_o, 2))
    assert np.isfinite(host(logp)).all()
    loss, lse, lse_rest = lp.lp_distill_top(student, ids, logp, rest)
    want = O.distill_top(z, host(ids), host(logp), host(rest), None, 1.0)
    assert np.isfinite(want[0]).all()
    close(host(loss), want[0], 2 * SUM * 2 + 2.0 ** -24 * np.abs(want[0]))
    # by itself: KL over the allowed tokens
    p = np.where(allowed, np.exp(t64 - np.where(allowed, t64, -np.inf).max(1, keepdims=True)), 0)
    p /= p.sum(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        kl = np.where(allowed, p * (np.log(p) - O.log_softmax(z)), 0).sum(1)
    close(host(loss), kl, 1e-4)
    g = torch.ones(T, device="cuda")
    d = lp.lp_distill_top_backward(student, ids, logp, rest, None, 1.0, lse, lse_rest, g)
    ref = O.distill_top_backward(z, host(ids), host(logp), host(rest), None, 1.0, np.ones(T))
    close(host(d), ref, grad_tol(z, host(ids), host(logp), host(rest), 1.0, np.ones(T), ref, "fp32"))
