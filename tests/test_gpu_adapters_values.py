"""Adapters on values that are hard to hold: infinities among the operands, all 24 bits of v and u, and
a wide range of them."""
import numpy as np
import pytest
import torch

from oracle import tokens as ref
from test_gpu_adapters import backward, forward, make, numbers, sizes
from token_harness import DTYPES, assert_near

pytestmark = pytest.mark.gpu


def whole(seed, most, *shape, dtype):
    """Whole numbers -most .. most: every product and sum below is a whole number that fp32 holds exactly."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).to(dtype).cuda()


def make_whole(T, n, r, inner, outer, dt, wt):
    d, w = DTYPES[dt], DTYPES[wt]
    rng = np.random.default_rng(T)
    return dict(adapter=torch.from_numpy(rng.integers(-1, n, T).astype(np.int32)).cuda(), x=whole(1, 50, T, inner, dtype=d),
                a=whole(2, 3, n, r, inner, dtype=w), b=whole(3, 3, n, outer, r, dtype=w),
                scale=2.0 ** -torch.arange(n, device="cuda").float(), base=whole(4, 50, T, outer, dtype=d),
                d_out=whole(5, 50, T, outer, dtype=d), dx_base=whole(6, 50, T, inner, dtype=d))


def assert_same(got, want):
    """The oracle's numbers rounded once; infinities with their sign, NaN where it has NaN."""
    with np.errstate(over="ignore"):
        want = torch.from_numpy(want).to(got.dtype).cuda()
    other = (torch.isnan(got) != torch.isnan(want)) | ((got != want) & ~torch.isnan(want))
    assert not other.any(), (int(other.sum()), got[other][:4].tolist(), want[other][:4].tolist())


# rows of one kernel each, blocks of 16 rows, ranks beyond the ones a wave keeps, blocks of 32 rows
SIZES = [(24, 16, 64, 72), (1100, 16, 64, 72), (1100, 72, 64, 72), (4200, 40, 64, 72), (8200, 64, 64, 72)]


@pytest.mark.parametrize("dt,wt", [("f32", "f32"), ("f32", "f16"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,r,inner,outer", SIZES)
def test_infinite_weights(T, r, inner, outer, dt, wt):
    """inf * v is an infinity of v's sign (NaN where v is 0), however v is held."""
    s = make_whole(T, 3, r, inner, outer, dt, wt)
    inf = float("inf")
    s["b"][0, 5, 2], s["b"][1, 7, 0], s["b"][1, 7, 3], s["b"][2, outer - 1, r - 1] = inf, inf, -inf, -inf
    m = numbers(s)
    with np.errstate(invalid="ignore"):
        assert_same(forward(s), ref.adapters(m["x"], m["adapter"], m["a"], m["b"], m["scale"]))
        assert_same(forward(s, base=s["base"]), ref.adapters(m["x"], m["adapter"], m["a"], m["b"], m["scale"], m["base"]))
    s = make_whole(T, 3, r, inner, outer, dt, wt)
    s["a"][0, 2, 5], s["a"][1, 0, 7], s["a"][1, 3, 7], s["a"][2, r - 1, inner - 1] = inf, inf, -inf, -inf
    m = numbers(s)
    with np.errstate(invalid="ignore"):
        want = ref.adapters_backward(m["d_out"], m["x"], m["adapter"], m["a"], m["b"], m["scale"], m["dx_base"])
        assert_same(backward(s, dx_base=s["dx_base"])[0], want[0])


@pytest.mark.parametrize("dt,wt", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,r", [(300, 16), (300, 24), (300, 40), (900, 16), (900, 24), (900, 40)])
def test_infinite_activations_and_gradients(T, r, dt, wt):
    """An overflowed x or d_out: d_a and d_b of its adapter get infinities of the right sign."""
    inf, inner, outer = float("inf"), 64, 72
    for name, direct in (("x", 1), ("d_out", 2)):     # the gradient whose product it is an operand of
        s = make_whole(T, 3, r, inner, outer, dt, wt)
        first = [int(torch.nonzero(s["adapter"] == e)[3, 0]) for e in range(3)]
        s[name][first[0], 9], s[name][first[1], 11], s[name][first[1], 12] = inf, -inf, inf
        s[name][first[2], 63] = -inf
        m = numbers(s)
        with np.errstate(invalid="ignore"):
            want = ref.adapters_backward(m["d_out"], m["x"], m["adapter"], m["a"], m["b"], m["scale"])
        got = backward(s)
        for g, w in zip(got, want):
            assert_same(g, w)
        assert torch.isinf(got[direct]).any()


@pytest.mark.parametrize("dt,wt", [("f32", "f32"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("T", [300, 900])
@pytest.mark.parametrize("r", [4, 20, 40])
def test_gradients_of_single_rows_hold_all_of_v_and_u(T, r, dt, wt):
    """Each adapter has one row, whose v and u are an fp32 scale of 24 bits times powers of two: d_a = u x^T
    and d_b = d_out v^T are then fp32 numbers and have to be exact."""
    inner, outer = 72, 64
    rng = np.random.default_rng(T + r)
    s = make(T, T, r, inner, outer, dt, wt, "mixed", seed=970)
    s["adapter"] = torch.from_numpy(rng.permutation(T).astype(np.int32)).cuda()

    def powers(*shape, dtype):
        return torch.from_numpy(rng.choice([-1.0, 1.0], shape) * 2.0 ** rng.integers(-3, 4, shape)).to(dtype).cuda()

    x, d_out = (torch.zeros_like(s[n]) for n in ("x", "d_out"))
    for t in (x, d_out):                          # a row has one element, so v and u have one term
        at = torch.from_numpy(rng.integers(0, t.shape[1], T)).cuda()
        t[torch.arange(T, device="cuda"), at] = powers(T, dtype=t.dtype)
    s.update(x=x, d_out=d_out, a=powers(T, r, inner, dtype=DTYPES[wt]), b=powers(T, outer, r, dtype=DTYPES[wt]))
    m = numbers(s)
    want = ref.adapters_backward(m["d_out"], m["x"], m["adapter"], m["a"], m["b"], m["scale"])
    got = backward(s)
    for g, w in zip(got[1:], want[1:]):
        assert np.array_equal(g.double().cpu().numpy(), w)


# rows of one kernel each (forward), blocks of 16 rows, ranks beyond the ones a wave keeps, blocks of 32 rows
WIDE = [(40, 16), (1500, 16), (1500, 100), (4200, 32), (8200, 64)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,r", WIDE)
@pytest.mark.parametrize("m", [12, 20, 28])
def test_components_far_below_the_largest(T, r, m, dt):
    """v and u with one component 2^m above the others, which weights of zero keep out of the result."""
    s = make(T, 3, r, 64, 72, dt, dt, "runs", seed=950 + m)
    up, down = 2.0 ** (m // 2), 2.0 ** -(m // 2)
    t = dict(s, a=s["a"] * down, b=s["b"] * up)
    t["a"][:, 0], t["b"][:, :, 0] = s["a"][:, 0] * up, 0
    mm, dtype = numbers(t), s["x"].dtype
    z = sizes(mm)
    want = ref.adapters(mm["x"], mm["adapter"], mm["a"], mm["b"], mm["scale"])
    size = ref.adapters(z["x"], mm["adapter"], z["a"], z["b"], z["scale"])
    assert_near(forward(t), want, dtype, (64 + r + 16) * 2.0 ** -23 * size)
    t = dict(s, b=s["b"] * down, a=s["a"] * up)
    t["b"][:, :, 0], t["a"][:, 0] = s["b"][:, :, 0] * up, 0
    mm = numbers(t)
    z = sizes(mm)
    args = [(q["d_out"], q["x"], mm["adapter"], q["a"], q["b"], q["scale"]) for q in (mm, z)]
    want, size = ref.adapters_backward(*args[0]), ref.adapters_backward(*args[1])
    for g, w, e, terms, of in zip(backward(t), want, size, (72 + r, 72 + T, 64 + T), (dtype, torch.float32, torch.float32)):
        assert_near(g, w, of, (terms + 16) * 2.0 ** -23 * e)


@pytest.mark.parametrize("dt,wt", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,r", [(24, 2), (1100, 2), (1500, 40), (1500, 90), (8200, 64)])
def test_products_that_cancel(T, r, dt, wt):
    """Two ranks with v = s p and v = s p q, of weights q and -1: what is left of s p q - s p q are the roundings of v and
    of the sum of the two products, in three parts each at most: 8 times 2^-23 of the products' sizes."""
    n, inner, outer, q = 5, 64, 72, 1 + 2.0 ** -7
    s = make(T, n, r, inner, outer, dt, wt, "mixed", seed=980)
    rng = np.random.default_rng(T + r)
    one, other = rng.permutation(r)[:2]

    def single(t):
        t.zero_()
        at = torch.from_numpy(rng.integers(0, t.shape[1], T)).cuda()
        t[torch.arange(T, device="cuda"), at] = torch.from_numpy(2.0 ** rng.integers(-3, 4, T)).to(t.dtype).cuda()

    for name in ("x", "d_out"):
        single(s[name])
    for a, b in (((1, q), (q, -1)), ((q, -1), (1, q))):     # of the forward; of the backward
        s["a"].zero_()
        s["b"].zero_()
        s["a"][:, one], s["a"][:, other] = a
        s["b"][:, :, one], s["b"][:, :, other] = b
        m = numbers(s)
        z, dtype = sizes(m), s["x"].dtype
        if a[0] == 1:
            assert_near(forward(s), np.zeros((T, outer)), dtype,
                        2.0 ** -20 * ref.adapters(z["x"], m["adapter"], z["a"], z["b"], z["scale"]))
        else:
            size = ref.adapters_backward(z["d_out"], z["x"], m["adapter"], z["a"], z["b"], z["scale"])[0]
            assert_near(backward(s)[0], np.zeros((T, inner)), dtype, 2.0 ** -20 * size)
