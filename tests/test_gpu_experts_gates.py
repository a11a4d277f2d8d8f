"""Large and infinite gates through the activations and their slopes, in every type.

The 16-bit types evaluate sigmoid(z) = 1 / (1 + 2^(-z log2 e)) with the hardware's exponential and reciprocal (1 unit in the
last place each); the exponent's argument is off by 2 roundings, so sigmoid(z) by (|z| + 5) 2^-23 of itself, and
gelu's z by 4 roundings more: (5 |z| + 5) 2^-23.
"""
import numpy as np
import pytest
import torch

import expert_offload_lru_amd as moe
from token_harness import DTYPES, assert_near, f64

pytestmark = pytest.mark.gpu


def run(gates, t, act):
    """hidden of gates with u = 1 (a reduction of one product, so that no other value enters), and d_pre for d_h = 1."""
    I = len(gates)
    g = torch.tensor(gates, device="cuda").to(t)
    w = torch.cat([g, torch.ones(I, dtype=t, device="cuda")]).reshape(1, 2 * I, 1)
    x, off = torch.ones(1, 1, dtype=t, device="cuda"), torch.tensor([0, 1], dtype=torch.int32).cuda()
    h, pre, d_pre = (torch.full((1, n), 7.0, dtype=t, device="cuda") for n in (I, 2 * I, 2 * I))
    moe.experts_hidden(x, off, w, h, activation=act, pre=pre)
    assert torch.equal(pre[0, I:], torch.ones_like(g)) and torch.equal(torch.nan_to_num(pre[0, :I]), torch.nan_to_num(g))
    again = torch.empty_like(h)
    moe.experts_hidden_backward(x, off, torch.ones(1, 1, I, dtype=t, device="cuda"), d_pre, hidden=again, activation=act, pre=pre)
    assert torch.equal(torch.nan_to_num(again, nan=3.0), torch.nan_to_num(h, nan=3.0))
    return f64(g), h[0], d_pre[0, :I], d_pre[0, I:]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_large_gates(dtype, act):
    t = DTYPES[dtype]
    big = [30.0, 89.0, 200.0, 6e4] + ([1e10, 1e30] if dtype != "f16" else [])
    g, h, dg, du = run(big + [-v for v in big], t, act)
    n = len(big)
    assert np.array_equal(f64(h[:n]), g[:n]) and np.array_equal(f64(du[:n]), g[:n]) and (f64(dg[:n]) == 1).all()
    for v in (h[n + 1:], dg[n + 1:], du[n + 1:]):   # from -89 on
        assert (v.float().abs() < 1e-30).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gates_down_to_the_last_normal_sigmoid(dtype, act):
    t = DTYPES[dtype]
    g, h, dg, du = run(np.concatenate([np.linspace(-87, 87, 349), np.linspace(-7, 7, 141)]).tolist(), t, act)
    if act == "silu":
        z, dz = g, np.ones_like(g)
    else:
        c = np.sqrt(8 / np.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g * g)
    p = 1 / (1 + np.exp(-np.clip(z, -700, 700)))
    e = (5 * np.abs(z) + 5) * 2.0 ** -23
    # below 2^-126 a sigmoid may be cut to 0
    tiny = np.where(p < 2.0 ** -125, p, 0.0)
    a = np.where(np.abs(z) > 600, np.maximum(g, 0), g * p)   # without tanh's cancellation
    assert_near(h, a, t, np.abs(a) * e + np.abs(g) * tiny)
    assert_near(du, a, t, np.abs(a) * e + np.abs(g) * tiny)
    # slope = p + a (1 - p) z': 1 - p adds a rounding of p near 1 and p's own error, which is p (1 - p) |z| of them
    q = 1 / (1 + np.exp(np.clip(z, -700, 700)))
    err = p * e + np.abs(a) * dz * (2 * q * e + 2.0 ** -23 * (q < 0.75)) + (np.abs(g) * dz + 1) * tiny
    slope = p + a * q * dz
    assert_near(dg, slope, t, err + 4 * 2.0 ** -24 * (p + np.abs(a) * q * dz))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_infinite_gates_are_not_hidden(dtype, act):
    """As the formulas in fp32: an infinite gate is infinite or NaN (inf times 0), and its slope NaN; other gates are as alone."""
    t, inf = DTYPES[dtype], float("inf")
    _, h, dg, du = run([inf, -inf, float("nan"), 2.0, -1.0], t, act)
    _, h1, dg1, du1 = run([2.0, -1.0], t, act)
    assert h[0] == inf and du[0] == inf and torch.isnan(h[1:3]).all() and torch.isnan(du[1:3]).all() and torch.isnan(dg[:3]).all()
    assert torch.equal(h[3:], h1) and torch.equal(dg[3:], dg1) and torch.equal(du[3:], du1)
