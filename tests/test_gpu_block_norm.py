"""Block norms on the GPU against float64 (oracle/experts.py).

Tolerances: a row's mean square is a sum of positive terms added in a tree (at most 32 in a lane, then 6 + 4 steps), so its inverse
root is off by 2^-19 at most (64 roundings of 2^-24 and half of them by the root: 2^-19 leaves room for the rest); a
product chain adds 8 roundings.
"""
import numpy as np
import pytest
import torch

import expert_offload_lru_amd as moe
from oracle import experts as o
from token_harness import DTYPES, assert_near, f64, place, randn

pytestmark = pytest.mark.gpu
R5 = 2.0 ** -19

WIDTHS = [1, 7, 64, 500, 513, 770, 1024, 2048, 2049, 4096, 5000, 8192, 8200, 16384]
PARTS = [(1, 1, 1, 1), (1, 0, 0, 1), (0, 1, 0, 0), (1, 0, 1, 0), (0, 0, 0, 1), (0, 1, 1, 1)]


def params(H, R, post, gate, alpha, pre, per):
    p = {}
    if post:
        p["w_post"] = randn(11, H) + 1
    if gate:
        p["gate"] = randn(12, -(-R // per), H)
        p["rows_per_gate"] = per
    if alpha:
        p["alpha"] = randn(13, H)
    if pre:
        p["w_pre"] = randn(14, H) + 1
    return p


def oracle_of(p):
    q = {n: f64(v) for n, v in p.items() if n != "rows_per_gate"}
    if "rows_per_gate" in p:
        q["per"] = p["rows_per_gate"]
    return q


def forward(x, y, p, ld=None, offset=0, eps=1e-6):
    R, H = x.shape
    new = lambda: place(torch.full((R, H), 7.0, dtype=x.dtype).cuda(), ld or H, offset)  # noqa: E731
    out, normed, stats = new() if y is not None else None, new() if "w_pre" in p else None, torch.full((R, 2), 7.0, device="cuda")
    moe.block_norm(x, y, out, normed=normed, stats=stats, eps=eps, **p)
    return out, normed, stats


def check_forward(x, y, p, got, eps=1e-6):
    out, normed, stats = got
    q = oracle_of(p)
    ro, rn, ry, rr = o.norm(f64(x), None if y is None else f64(y), eps=eps, **q)
    size = np.abs(f64(x)) if y is None else o.norm(np.abs(f64(x)), np.abs(f64(y)), eps=eps,
                                                  **{n: v if n == "per" else np.abs(v) for n, v in q.items()})[0]
    if out is not None:
        assert_near(out, ro, x.dtype, R5 * size)
    s = f64(stats)
    assert (np.abs(s[:, 0] - ry) <= R5 * ry).all()
    # out's own error, against the root of its mean square
    e = R5 * (1 + np.sqrt(np.mean(size ** 2, 1, keepdims=True)) * (rr[:, None] if normed is not None else 0))
    if normed is not None:
        assert (np.abs(s[:, 1] - rr) <= e[:, 0] * rr).all()
        assert_near(normed, rn, x.dtype, e * np.abs(rn) + np.abs(q["w_pre"]) * rr[:, None] * R5 * size)
    else:
        assert (s[:, 1] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", WIDTHS)
def test_forward(H, dtype):
    t = DTYPES[dtype]
    for R, per in ((1, 1), (3, 2), (13, 5)):
        x, y = randn(1, R, H, dtype=t, std=3.0), randn(2, R, H, dtype=t)
        for parts in PARTS if R == 3 else PARTS[:1]:
            p = params(H, R, *parts, per)
            check_forward(x, y, p, forward(x, y, p))
        p = params(H, R, 0, 0, 0, 1, 1)
        check_forward(x, None, p, forward(x, None, p))


def grads(p, H):
    return {"d_" + n: torch.full_like(v, 7.0) for n, v in p.items() if n != "rows_per_gate"}


def check_backward(x, y, p, R, H, with_out=True, with_normed=True):
    t = x.dtype
    stats = forward(x, y, p)[2]
    d_out = randn(21, R, H, dtype=t) if with_out else None
    d_n = randn(22, R, H, dtype=t) if with_normed and "w_pre" in p else None
    d_x, d_y = torch.full_like(x, 7.0), None if y is None else torch.full_like(x, 7.0)
    g = grads(p, H)
    moe.block_norm_backward(d_out, x, y, stats, d_x, d_y, d_normed=d_n, **p, **g)
    q, s = oracle_of(p), f64(stats)
    args = lambda f: (None if d_out is None else f(f64(d_out)), None if d_n is None else f(f64(d_n)), f(f64(x)),  # noqa: E731
                      None if y is None else f(f64(y)))
    ref = o.norm_backward(*args(lambda v: v), s[:, 0], s[:, 1], **q)
    # the same with every term's size: D's subtraction added instead
    big = sizes(*args(np.abs), s[:, 0], s[:, 1], **{n: v if n == "per" else np.abs(v) for n, v in q.items()})
    assert_near(d_x, ref["d_x"], t, R5 * big["d_x"])
    if y is not None:
        assert_near(d_y, ref["d_y"], t, R5 * big["d_y"])
    for n, v in g.items():
        want = ref.get(n, np.zeros(v.shape))
        assert_near(v, want, torch.float32, (R5 + R * 2.0 ** -24) * big.get(n, 0.0))
    return d_x, d_y, g


def sizes(d_out, d_n, x, y, r_y, r_o, w_post=None, gate=None, per=1, alpha=None, w_pre=None):
    """norm_backward with every subtraction added: what roundings are relative to."""
    R, H = x.shape
    y = np.zeros((R, H)) if y is None else y
    a, g = 1.0 if alpha is None else alpha, 1.0 if gate is None else gate[np.arange(R) // per]
    wp = 1.0 if w_post is None else w_post
    ry = np.ones((R, 1)) if w_post is None else r_y.reshape(R, 1)
    ro = r_o.reshape(R, 1)
    z = y * ry
    out = x * a + g * wp * z
    D, got = np.zeros((R, H)) if d_out is None else d_out, {}
    if d_n is not None:
        t = w_pre * d_n
        D = D + ro * t + out * ro ** 3 * np.mean(t * out, 1, keepdims=True)
        got["d_w_pre"] = np.sum(d_n * out * ro, 0)
    c = g * wp * D
    got["d_x"] = a * D
    got["d_y"] = c if w_post is None else ry * c + y * ry ** 3 * np.mean(c * y, 1, keepdims=True)
    got["d_alpha"], got["d_w_post"] = np.sum(D * x, 0), np.sum(g * D * z, 0)
    dg = wp * D * z
    got["d_gate"] = np.stack([dg[i:i + per].sum(0) for i in range(0, R, per)])
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", WIDTHS)
def test_backward(H, dtype):
    t = DTYPES[dtype]
    for R, per in ((1, 1), (5, 2), (21, 21)):
        x, y = randn(1, R, H, dtype=t, std=3.0), randn(2, R, H, dtype=t)
        for parts in PARTS if R == 5 else PARTS[:1]:
            check_backward(x, y, params(H, R, *parts, per), R, H)
        check_backward(x, None, params(H, R, 0, 0, 0, 1, 1), R, H)
        check_backward(x, y, params(H, R, 1, 1, 1, 1, per), R, H, with_out=False)
        check_backward(x, y, params(H, R, 1, 1, 1, 1, per), R, H, with_normed=False)


@pytest.mark.parametrize("R,per", [(1200, 1), (1200, 2), (1200, 3), (1200, 7), (1200, 64), (1200, 500), (1200, 1200), (1200, 5000),
                                   (4200, 9), (4200, 8), (513, 512), (600, 599)])
@pytest.mark.parametrize("H", [64, 1000])
def test_gates_of_many_lengths(R, per, H):
    """A gate's rows within a chunk of rows, over several, and the last one short."""
    x, y = randn(1, R, H, dtype=torch.bfloat16), randn(2, R, H, dtype=torch.bfloat16)
    check_backward(x, y, params(H, R, 1, 1, 1, 1, per), R, H)


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_in_place(dtype):
    t = DTYPES[dtype]
    R, H = 40, 200
    x, y = randn(1, R, H, dtype=t), randn(2, R, H, dtype=t)
    p = params(H, R, 1, 1, 1, 1, 7)
    out, normed, stats = forward(x, y, p)
    for ld, at in ((H + 8, 0), (H + 1, 1), (H + 3, 5)):
        got = forward(place(x, ld, at), place(y, ld, at), p, ld, at)
        assert all(torch.equal(a, b) for a, b in zip(got, (out, normed, stats)))
    x2, y2 = x.clone(), y.clone()
    moe.block_norm(x2, y2, x2, normed=y2, **p)
    assert torch.equal(x2, out) and torch.equal(y2, normed)
    d, dn = randn(3, R, H, dtype=t), randn(4, R, H, dtype=t)
    d_x, d_y = torch.empty_like(x), torch.empty_like(x)
    moe.block_norm_backward(d, x, y, stats, d_x, d_y, d_normed=dn, **p)
    for ld, at in ((H + 8, 0), (H + 1, 1)):
        a, b = place(d_x, ld, at).fill_(7), place(d_y, ld, at).fill_(7)
        moe.block_norm_backward(*(place(v, ld, at) for v in (d, x, y)), stats, a, b, d_normed=place(dn, ld, at), **p)
        assert torch.equal(a, d_x) and torch.equal(b, d_y)
    d2, dn2 = d.clone(), dn.clone()
    moe.block_norm_backward(d2, x, y, stats, d2, dn2, d_normed=dn2, **p)
    assert torch.equal(d2, d_x) and torch.equal(dn2, d_y)


def test_rows_of_zeros_and_large_values():
    H = 96
    x = torch.zeros(4, H, device="cuda")
    x[1], x[2], x[3] = 1e18, 1e-18, float("nan")
    normed, stats = torch.empty_like(x), torch.empty(4, 2, device="cuda")
    moe.block_norm(x, None, None, w_pre=torch.ones(H, device="cuda"), normed=normed, stats=stats)
    assert not normed[0].any() and torch.allclose(normed[1], torch.ones(H, device="cuda")) and torch.isnan(normed[3]).all()
    assert abs(float(stats[0, 1]) - 1000) < 1e-3 and torch.allclose(normed[2], torch.full((H,), 1e-15, device="cuda"))


def test_no_rows():
    H = 64
    x = torch.empty(0, H, device="cuda")
    p = params(H, 0, 1, 0, 1, 1, 1)
    moe.block_norm(x, x.clone(), x.clone(), normed=x.clone(), **p)
    g = grads(p, H)
    moe.block_norm_backward(x, x.clone(), x.clone(), torch.empty(0, 2, device="cuda"), x.clone(), x.clone(), d_normed=x.clone(), **p, **g)
    assert not any(v.any() for v in g.values())


def test_same_bits_again():
    R, H = 3000, 300
    x, y, d = (randn(i, R, H, dtype=torch.bfloat16) for i in (1, 2, 3))
    p = params(H, R, 1, 1, 1, 1, R)
    stats = forward(x, y, p)[2]
    runs = []
    for _ in range(3):
        g = grads(p, H)
        d_x, d_y = torch.empty_like(x), torch.empty_like(x)
        moe.block_norm_backward(d, x, y, stats, d_x, d_y, d_normed=d, **p, **g)
        runs.append([d_x, d_y, *g.values()])
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("H", [200, 9000])
def test_without_out_or_stats(H):
    """normed alone, stats alone, out alone: the same bits as together."""
    R = 9
    x, y = randn(1, R, H, dtype=torch.bfloat16), randn(2, R, H, dtype=torch.bfloat16)
    p = params(H, R, 1, 1, 1, 1, 4)
    out, normed, stats = forward(x, y, p)
    a, b, c = torch.empty_like(x), torch.empty(R, 2, device="cuda"), torch.empty_like(x)
    moe.block_norm(x, y, None, normed=a, **p)
    moe.block_norm(x, y, None, stats=b, **{**p, "w_pre": None})
    moe.block_norm(x, y, c, **{**p, "w_pre": None})
    assert torch.equal(a, normed) and torch.equal(c, out) and torch.equal(b[:, 0], stats[:, 0]) and not b[:, 1].any()


def test_rows_far_apart():
    """Offsets past 31 bits between rows."""
    H, ld = 72, (1 << 30) + 3
    x, y = randn(1, 3, H, dtype=torch.float16), randn(2, 3, H, dtype=torch.float16)
    p = params(H, 3, 1, 0, 0, 1, 1)
    out, normed, stats = forward(x, y, p)
    # a buffer each: column ranges of one matrix count as overlapping
    far = [torch.empty(3 * ld, dtype=torch.float16, device="cuda").view(3, ld)[:, :H] for _ in range(4)]
    far[0].copy_(x), far[1].copy_(y)
    moe.block_norm(far[0], far[1], far[0], normed=far[1], **p)
    assert torch.equal(far[0], out) and torch.equal(far[1], normed)
    far[0].copy_(x), far[1].copy_(y), far[2].copy_(out), far[3].copy_(normed)
    d_x, d_y = torch.empty_like(x), torch.empty_like(x)
    moe.block_norm_backward(out, x, y, stats, d_x, d_y, d_normed=normed, **p)
    moe.block_norm_backward(far[2], far[0], far[1], stats, far[2], far[3], d_normed=far[3], **p)
    assert torch.equal(far[2], d_x) and torch.equal(far[3], d_y)


@pytest.mark.parametrize("size", [1e15, 1e-15, 1e18])
def test_backward_of_rows_of_any_size(size):
    """r^3 of such rows is outside fp32's range."""
    R, H = 7, 200
    x, y = randn(1, R, H) * size, randn(2, R, H) * size
    check_backward(x, y, params(H, R, 1, 1, 1, 1, 3), R, H)
    check_backward(x, None, params(H, R, 0, 0, 0, 1, 1), R, H)
