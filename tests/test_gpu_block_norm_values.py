"""Block norms of rows of any size, from the largest numbers of a type down to those that eps does not hold up, against
float64 (oracle/experts.py).  Tolerances as in test_gpu_block_norm.py: a row that is summed again is scaled by a power of two,
which rounds nothing; an inverse root below 2^-126 has 21 bits and more, so its rounding stays under 2^-21.
"""
import pytest
import torch

import expert_offload_lru_amd as moe
from test_gpu_block_norm import PARTS, check_backward, check_forward, forward, params
from token_harness import DTYPES, place, randn

pytestmark = pytest.mark.gpu

WIDE = ["f32", "bf16"]   # types that hold 1e37
# one wave a row and more, and, at 700 and 1000, two rows that share a barrier
WIDTHS = [96, 512, 700, 1000, 2048, 2100, 4096, 8192, 16384]
# squares over and under fp32's range beside ordinary ones, in every place of a workgroup's rows
SIZES = [1.0, 1e18, 1e37, 1e-3, 3e30, 1.0, 1e19, 1e25, 2.0, 1.0, 1e37]


def rows(seed, H, sizes, t):
    return (randn(seed, len(sizes), H) * torch.tensor(sizes, device="cuda")[:, None]).to(t)


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("H", WIDTHS)
def test_forward_of_large_rows(H, dtype):
    t, R = DTYPES[dtype], len(SIZES)
    x, y = rows(1, H, SIZES, t), rows(2, H, SIZES[::-1], t)
    for parts in PARTS:
        p = params(H, R, *parts, 3)
        check_forward(x, y, p, forward(x, y, p))
    p = params(H, R, 0, 0, 0, 1, 1)
    got = forward(x, None, p)
    check_forward(x, None, p, got)
    # a row is the same beside any others
    for i in range(R):
        alone = forward(x[i:i + 1], None, p)
        assert torch.equal(alone[1], got[1][i:i + 1]) and torch.equal(alone[2], got[2][i:i + 1])


@pytest.mark.parametrize("H", WIDTHS)
def test_forward_of_small_rows_without_eps(H):
    sizes = [1.0, 1e-25, 1e-36, 1e-3, 1e18, 1.0, 1e-20, 1e-12, 1e-15, 2e-16, 1e30]
    x, y = rows(1, H, sizes, torch.float32), rows(2, H, sizes[::-1], torch.float32)
    for eps in (0.0, 1e-32):
        for parts in PARTS:
            p = params(H, len(sizes), *parts, 3)
            check_forward(x, y, p, forward(x, y, p, eps=eps), eps=eps)
        p = params(H, len(sizes), 0, 0, 0, 1, 1)
        check_forward(x, None, p, forward(x, None, p, eps=eps), eps=eps)


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("H", [96, 700, 2048, 8192, 16384])
def test_backward_of_large_rows(H, dtype):
    t, R = DTYPES[dtype], len(SIZES)
    x, y = rows(1, H, SIZES, t), rows(2, H, SIZES[::-1], t)
    for with_out in (True, False):
        check_backward(x, y, params(H, R, 1, 1, 1, 1, 3), R, H, with_out=with_out)
    check_backward(x, None, params(H, R, 0, 0, 0, 1, 1), R, H)


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("H", [96, 1000, 4096])
def test_largest_rows(H, dtype):
    """Every value the type's largest or least number: normalised to 1 and -1."""
    t = DTYPES[dtype]
    x = torch.full((5, H), torch.finfo(t).max, dtype=t, device="cuda")
    x[1::2] *= -1
    x[4] = 0
    normed, stats = torch.empty_like(x), torch.empty(5, 2, device="cuda")
    moe.block_norm(x, None, None, w_pre=torch.ones(H, device="cuda"), normed=normed, stats=stats)
    want = torch.sign(x.float())
    assert ((normed.float() - want).abs() <= 2.0 ** -19 + torch.finfo(t).eps / 2).all() and not normed[4].any()
    r = 1 / x[0, 0].double()
    assert ((stats[:4, 1].double() - r).abs() <= 2.0 ** -19 * r).all()


@pytest.mark.parametrize("H", [96, 700, 1000, 2048, 16384])
def test_rows_beside_infinite_ones(H):
    """An infinite or NaN row changes no other: the rows beside it have the same bits."""
    t = torch.float32
    x, y = rows(1, H, SIZES, t), rows(2, H, SIZES[::-1], t)
    p = params(H, len(SIZES), 1, 1, 1, 1, 3)
    want = forward(x, y, p)
    u, v = x.clone(), y.clone()
    u[1, 5], v[4, 0], u[7, H - 1] = float("inf"), float("nan"), float("-inf")
    got = forward(place(u, H + 3, 1), place(v, H + 3, 1), p)
    same = [i for i in range(len(SIZES)) if i not in (1, 4, 7)]
    for a, b in zip(got, want):
        assert torch.equal(a[same], b[same])
    assert (got[2][[1, 7], 1] == 0).all() and torch.isnan(got[2][4]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [96, 1000, 2100, 9000])
@pytest.mark.parametrize("pre", ["no second norm", "its gradient not given"])
def test_infinities_that_a_gradient_does_not_depend_on(H, dtype, pre):
    """Without the second norm's gradient D = d_out: d_y does not see x, d_x sees neither, and without w_post d_y does not
    see y."""
    t, R = DTYPES[dtype], 9
    x, y, d_out = (randn(i, R, H, dtype=t) for i in (1, 2, 21))
    u, v = x.clone(), y.clone()
    u[2, 5], u[4], u[6, H - 1] = float("inf"), float("-inf"), float("nan")
    v[1, 0], v[4, 7], v[8] = float("nan"), float("inf"), float("-inf")
    for post, gate, alpha in ((1, 1, 1), (1, 0, 0), (0, 1, 1), (0, 0, 1), (0, 0, 0)):
        p = params(H, R, post, gate, alpha, pre != "no second norm", 4)

        def grads(x, y):
            d_x, d_y = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
            moe.block_norm_backward(d_out, x, y, forward(x, y, p)[2], d_x, d_y, **p)
            return d_x, d_y

        want = grads(x, y)
        for given in ((u, y), (x, v), (u, v)):
            d_x, d_y = grads(*given)
            assert torch.equal(d_x, want[0])
            rows = [0, 2, 3, 5, 6, 7] if post and given[1] is v else list(range(R))
            assert torch.equal(d_y[rows], want[1][rows])
