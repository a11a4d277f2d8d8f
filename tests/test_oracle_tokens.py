"""Pins of oracle/tokens.py: hand-worked values and derivatives by differences (CPU)."""
import numpy as np
import pytest

from oracle import tokens as ref


def test_order_by_hand():
    ids = np.array([[2, 0], [-1, 2], [0, 9], [2, 2]])
    o = ref.order(ids, 3)
    assert o["offsets"].tolist() == [0, 2, 2, 6]
    assert o["src"].tolist() == [1, 4, 0, 3, 6, 7, -1, -1]
    assert o["expert"].tolist() == [0, 0, 2, 2, 2, 2, -1, -1]
    assert o["pos"].tolist() == [[2, 0], [-1, 3], [1, -1], [4, 5]]
    x = np.arange(4.0)[:, None]
    assert ref.dispatch(x, o, np.full((8, 1), 9.0))[:, 0].tolist() == [0, 2, 0, 1, 3, 3, 9, 9]


def test_combine_by_hand():
    rows, pos, gate = np.array([[1.0], [10.0], [100.0]]), np.array([[2, 0], [-1, 1], [-1, -1]]), np.array([[.5, 2], [7, 3], [1, 1]])
    assert ref.combine(rows, pos, gate, np.array([[1.0], [2.0], [3.0]]))[:, 0].tolist() == [53.0, 32.0, 3.0]
    assert ref.combine(rows, pos)[:, 0].tolist() == [101.0, 10.0, 0.0]
    d_rows, d_gate = ref.combine_backward(np.array([[2.0], [3.0], [4.0]]), rows, pos, gate, np.zeros((3, 1)))
    assert d_rows[:, 0].tolist() == [4.0, 9.0, 1.0]
    assert d_gate.tolist() == [[200.0, 2.0], [0.0, 30.0], [0.0, 0.0]]


def test_adapters_by_hand():
    a, b = np.array([[[1.0, 2.0]], [[0.0, 1.0]]]), np.array([[[3.0]], [[5.0]]])
    x, scale = np.array([[1.0, 1.0], [2.0, 4.0], [9.0, 9.0]]), np.array([2.0, 0.5])
    assert ref.adapters(x, np.array([0, 1, -1]), a, b, scale, np.ones((3, 1)))[:, 0].tolist() == [19.0, 11.0, 1.0]


@pytest.mark.parametrize("name", ["x", "a", "b"])
def test_adapter_gradients_by_differences(name):
    rng = np.random.default_rng(3)
    s = dict(x=rng.normal(size=(7, 5)), a=rng.normal(size=(3, 2, 5)), b=rng.normal(size=(3, 4, 2)))
    which, scale, w = np.array([0, 2, -1, 2, 0, 5, 2]), rng.normal(size=3), rng.normal(size=(7, 4))
    g = dict(zip("xab", ref.adapters_backward(w, s["x"], which, s["a"], s["b"], scale)))
    d = rng.normal(size=s[name].shape)

    def loss(sign):
        t = dict(s, **{name: s[name] + sign * d})
        return (ref.adapters(t["x"], which, t["a"], t["b"], scale) * w).sum()

    assert abs((loss(1) - loss(-1)) / 2 - (g[name] * d).sum()) < 1e-10
