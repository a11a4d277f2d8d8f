"""Pins of oracle/experts.py: worked numbers, and gradients against differences."""
import numpy as np
import pytest

from oracle import experts as o


def test_encode_by_hand():
    x = np.zeros((3, 40))
    x[0, :4] = [127.0, -1.0, 0.5, 1.5]        # scale 1: halves go to the even number
    x[0, 32:34] = [1.0, -0.009]               # a block of 8 columns, scale 2^-6
    x[1, 0] = 127.5                           # rounds to 128: scale 2
    x[2, 3], x[2, 35] = np.inf, 2.0 ** -140
    codes, scales = o.encode(x)
    assert scales.tolist() == [[133, 127], [134, 0], [255, 0]]
    assert codes[0, :4].tolist() == [127, -1, 0, 2] and codes[0, 32:34].tolist() == [64, -1]
    assert codes[1, 0] == 64 and not codes[2].any()
    v = o.decode(codes, scales)
    assert np.isnan(v[2, :32]).all() and not v[2, 32:].any() and v[0, 3] == 2.0 and v[0, 33] == -2.0 ** -6


def test_values_are_off_by_half_a_step():
    x = np.random.default_rng(1).standard_normal((20, 70)) * 10.0 ** np.random.default_rng(2).integers(-9, 9, (20, 1))
    codes, scales = o.encode(x)
    step = 2.0 ** (scales[:, np.arange(70) // 32] - 133)
    assert (np.abs(o.decode(codes, scales) - x) <= step / 2).all()
    tops = np.stack([np.abs(codes[:, i:i + 32]).max(1) for i in (0, 32, 64)], 1)
    assert (tops >= 64).all() and (tops <= 127).all()


def test_segments_of_odd_offsets():
    assert o.segments([0, 2, 2, 5], 9) == [(0, 0, 2), (1, 2, 2), (2, 2, 5)]
    assert o.segments([-3, 7, 4, 99], 9) == [(0, 0, 7), (1, 7, 7), (2, 7, 9)]


def _difference(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_block_gradients_by_differences(kind):
    rng = np.random.default_rng(3)
    R, H, I, E, off = 7, 5, 4, 3, np.array([0, 3, 3, 6])
    x, w, wd = rng.standard_normal((R, H)), rng.standard_normal((E, 2 * I, H)), rng.standard_normal((E, H, I))
    t = rng.standard_normal((R, H)) * (np.arange(R) < 6)[:, None]

    def f(x, w, wd):
        h, _ = o.hidden(x, off, w, kind, np.zeros((R, I)), np.zeros((R, 2 * I)))
        return np.sum(o.product(h, off, wd, np.zeros((R, H))) * t)

    h, pre = o.hidden(x, off, w, kind, np.zeros((R, I)), np.zeros((R, 2 * I)))
    d_pre, again, _ = o.hidden_backward(t, off, wd, pre, kind, np.zeros((R, 2 * I)), np.zeros((R, I)))
    assert np.allclose(again, h)
    d_x, d_w = o.product_backward(d_pre, x, off, w, np.zeros((R, H)))
    d_wd = o.product_backward(t, h, off, wd, np.zeros((R, I)))[1]
    for k, (v, g) in enumerate(((x, d_x), (w, d_w), (wd, d_wd))):
        d = rng.standard_normal(v.shape)
        args = [x, w, wd]
        num = _difference(lambda z: f(*args[:k], z, *args[k + 1:]), v, d)
        assert abs(num - np.sum(g * d)) <= 1e-6 * max(1, abs(num))


@pytest.mark.parametrize("post,gate,alpha,pre", [(1, 1, 1, 1), (0, 1, 0, 1), (1, 0, 1, 0), (0, 0, 0, 1)])
def test_norm_gradients_by_differences(post, gate, alpha, pre):
    rng = np.random.default_rng(4)
    R, H, per = 5, 6, 2
    v = dict(x=rng.standard_normal((R, H)), y=rng.standard_normal((R, H)))
    if post:
        v["w_post"] = rng.standard_normal(H)
    if gate:
        v["gate"] = rng.standard_normal((3, H))
    if alpha:
        v["alpha"] = rng.standard_normal(H)
    if pre:
        v["w_pre"] = rng.standard_normal(H)
    t, s = rng.standard_normal((R, H)), rng.standard_normal((R, H))

    def f(**v):
        out, normed, _, _ = o.norm(**v, per=per)
        return np.sum(out * t) + (np.sum(normed * s) if pre else 0)

    _, _, r_y, r_o = o.norm(**v, per=per)
    g = o.norm_backward(t, s if pre else None, v["x"], v["y"], r_y, r_o, per=per,
                        **{n: v[n] for n in v if n not in "xy"})
    for n in v:
        d = rng.standard_normal(v[n].shape)
        num = _difference(lambda z: f(**{**v, n: z}), v[n], d)
        assert abs(num - np.sum(g["d_" + n] * d)) <= 1e-6 * max(1, abs(num)), n


def test_norm_by_hand():
    out, normed, r_y, r_o = o.norm(np.array([[3.0, 4.0]]), w_pre=np.array([1.0, 2.0]), eps=0)
    assert np.allclose(normed, np.array([[3.0, 8.0]]) / np.sqrt(12.5)) and r_y[0] == 0
    out, normed, r_y, _ = o.norm(np.array([[1.0, 1.0]]), np.array([[3.0, 4.0]]), w_post=np.ones(2), alpha=np.array([2.0, 0.0]),
                                 gate=np.array([[1.0, -1.0]]), eps=0)
    assert np.allclose(out, [[2 + 3 / np.sqrt(12.5), -4 / np.sqrt(12.5)]]) and normed is None
