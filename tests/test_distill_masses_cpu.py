"""The oracle of distillation on entries whose mass is nothing in fp32."""
import numpy as np
import pytest

from oracle import lp_oracle as O


@pytest.mark.parametrize("t", [-110.0, -800.0, -1e9, -3.4e38, -np.inf])
def test_entries_without_mass_add_nothing(t):
    z = np.array([[0.0, 1.0, -np.inf, 2.0], [0.0, 1.0, -np.inf, -np.inf]])
    ids, lp = np.array([[1, 2], [0, 1]]), np.array([[np.log(0.4), t], [np.log(0.4), np.log(0.3)]])
    rest = np.array([np.log(0.6), t])
    loss, lse, lse_rest = O.distill_top(z, ids, lp, rest, None, 1.0)
    q = np.exp(z[0] - lse[0])
    assert np.isclose(loss[0], 0.4 * np.log(0.4 / q[1]) + 0.6 * np.log(0.6 / (q[0] + q[3])))
    q = np.exp(z[1] - lse[1])
    assert np.isclose(loss[1], 0.4 * np.log(0.4 / q[0]) + 0.3 * np.log(0.3 / q[1])) and lse_rest[1] == -np.inf
    d = O.distill_top_backward(z, ids, lp, rest, None, 1.0, np.ones(2))
    assert np.isfinite(d).all() and np.allclose(d[1, :2], [0.7 * q[0] - 0.4, 0.7 * q[1] - 0.3])


def test_a_tiny_mass_is_one():
    z = np.array([[0.0, 1.0, -np.inf], [0.0, 1.0, -np.inf]])
    loss = O.distill_top(z, np.array([[2, 0], [0, 1]]), np.array([[-100.0, -0.1], [-1.0, -1.0]]), np.array([-np.inf, -100.0]),
                         None, 1.0)[0]
    assert (loss == np.inf).all()
    loss = O.distill_top(z, np.array([[2, 0]] * 2), np.array([[np.nan, -0.1]] * 2), None, None, 1.0)[0]
    assert np.isnan(loss).all()
