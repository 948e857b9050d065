"""The oracle of beam selection where scores swallow the logits."""
import numpy as np

from oracle import lp_oracle as O


def test_within_a_beam_its_logits_decide():
    z = np.array([[0.0, 3.0, 1.0, 3.0, -np.inf], [5.0, 6.0, 7.0, 8.0, 9.0]])
    far = float(np.finfo(np.float32).min)
    s, p, y = O.beam_select(z, np.array([[far, far]]), 7, None, 0, 1.0)
    assert p.tolist() == [[0, 0, 0, 0, 1, 1, 1]] and y.tolist() == [[1, 3, 2, 0, 4, 3, 2]] and np.all(s == far)
    _, p, y = O.beam_select(z, np.array([[0.0, -np.inf]]), 4, None, 0, 1e30)
    assert p.tolist() == [[0] * 4] and y.tolist() == [[1, 3, 2, 0]]
