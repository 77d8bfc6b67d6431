"""The oracle of beam selection where logits are far from 0, pinned by hand."""
import numpy as np

from oracle import beam


def test_equal_logits_are_uniform_wherever_they_lie():
    for value in (0.0, 1e9, -1e18, 1e30, -4e37):
        s, p, t, _, _ = beam.select(np.full((1, 1, 8), value), np.array([[-1.0]]), 2)
        assert np.allclose(s, -1 - np.log(8.0), rtol=1e-15) and t.tolist() == [[0, 1]] and p.tolist() == [[0, 0]]


def test_fills_add_nothing():
    x = np.array([[[-1e30, np.log(3.0), -1e10, 0.0]]])
    s, _, t, _, _ = beam.select(x, np.array([[0.0]]), 4)
    assert np.allclose(np.exp(s[0, :2]), [0.75, 0.25]) and t.tolist() == [[1, 3, 2, 0]] and np.all(s[0, 2:] < -1e9)
