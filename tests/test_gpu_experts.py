"""Experts' feed-forward and rows kept in 8 bits on the GPU against float64 (oracle/experts.py).

Tolerances count roundings (tests/token_harness.py): a sum of n products in fp32 is off by at most
n 2^-23 of the sum of their sizes on the matrix cores, and a result is rounded once.  An activation adds
16 roundings of fp32 (2^-20 of its argument), and its slope is at most 1.13.
"""
import numpy as np
import pytest
import torch

import expert_offload_lru_amd as moe
from oracle import experts as o
from token_harness import DTYPES, assert_near, f64, place, randn

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -23


def offsets_of(seed, R, E, before=0, behind=0):
    """Uneven rows of E experts, some without any; the first and last rows belong to none."""
    rng = np.random.default_rng(seed)
    cuts = np.sort(rng.integers(before, R - behind + 1, E - 1)) if E > 1 else np.zeros(0, int)
    if E > 3:
        cuts[1] = cuts[0]
    return torch.tensor([before, *cuts.tolist(), R - behind], dtype=torch.int32).cuda()


def sevens(R, C, dtype, ld=None, offset=0):
    return place(torch.full((R, C), 7.0, dtype=dtype).cuda(), ld or C, offset)


def magnitude(x, off, w):
    """Sum over the reduction of |x| |w|."""
    return o.product(np.abs(f64(x)), f64(off).astype(int), np.abs(f64(w)), np.zeros((x.shape[0], w.shape[1])))


# rows, inner, outer, experts: one row and column on, around tiles of 256 rows and 128 or 256 columns and steps of 32
# and 64, odd widths (rows that no 16-byte load fits), few and many rows
SIZES = [(1, 1, 1, 1), (1, 64, 32, 3), (2, 129, 3, 2), (5, 8, 257, 7), (17, 200, 96, 16), (64, 256, 128, 1), (63, 72, 384, 70),
         (255, 64, 256, 1), (257, 128, 264, 2), (300, 65, 131, 5), (700, 520, 320, 3), (1100, 40, 33, 130), (515, 333, 250, 2)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,M,E", SIZES)
def test_product(R, K, M, E, dtype):
    t = DTYPES[dtype]
    x, w, off = randn(1, R, K, dtype=t), randn(2, E, M, K, dtype=t), offsets_of(3, R, E, before=R > 200, behind=R > 60)
    out = sevens(R, M, t)
    moe.experts_product(x, off, w, out)
    ref = o.product(f64(x), off.tolist(), f64(w), np.full((R, M), 7.0))
    assert_near(out, ref, t, (K + 1) * ULP * magnitude(x, off, w))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,M,E", SIZES)
def test_product_backward(R, K, M, E, dtype):
    t = DTYPES[dtype]
    x, w, off = randn(1, R, K, dtype=t), randn(2, E, M, K, dtype=t), offsets_of(3, R, E, before=R > 200, behind=R > 60)
    d_out = randn(4, R, M, dtype=t)
    d_x, d_w = sevens(R, K, t), torch.full((E, M, K), 7.0, device="cuda")
    moe.experts_product_backward(d_out, off, w, x=x, d_x=d_x, d_w=d_w)
    rx, rw = o.product_backward(f64(d_out), f64(x), off.tolist(), f64(w), np.full((R, K), 7.0))
    mx, mw = o.product_backward(np.abs(f64(d_out)), np.abs(f64(x)), off.tolist(), np.abs(f64(w)), np.zeros((R, K)))
    assert_near(d_x, rx, t, (M + 1) * ULP * mx)
    assert_near(d_w, rw, torch.float32, (R + 17) * ULP * mw)
    # one of the two alone gives the same
    x2, w2 = sevens(R, K, t), torch.full((E, M, K), 7.0, device="cuda")
    moe.experts_product_backward(d_out, off, w, d_x=x2)
    moe.experts_product_backward(d_out, off, w, x=x, d_w=w2)
    assert torch.equal(x2, d_x) and torch.equal(w2, d_w)


def hidden_slack(pre, mag, K):
    """Errors of g and u, and of act(g) u, before the last rounding."""
    I = pre.shape[1] // 2
    dg, du = np.split((K + 1) * ULP * mag, 2, 1)
    g, u = np.abs(pre[:, :I]), np.abs(pre[:, I:])
    return np.concatenate([dg, du], 1), (1.13 * dg + 2.0 ** -20 * g) * (u + du) + g * du


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,I,E", SIZES)
def test_hidden(R, K, I, E, dtype, act):
    t = DTYPES[dtype]
    x, w = randn(1, R, K, dtype=t), randn(2, E, 2 * I, K, dtype=t, std=K ** -0.5)
    off = offsets_of(3, R, E, before=R > 200, behind=R > 60)
    h, pre = sevens(R, I, t), sevens(R, 2 * I, t)
    moe.experts_hidden(x, off, w, h, activation=act, pre=pre)
    rh, rp = o.hidden(f64(x), off.tolist(), f64(w), act, np.full((R, I), 7.0), np.full((R, 2 * I), 7.0))
    sp, sh = hidden_slack(rp, magnitude(x, off, w), K)
    assert_near(pre, rp, t, sp)
    assert_near(h, rh, t, sh)
    bare = sevens(R, I, t)
    moe.experts_hidden(x, off, w, bare, activation=act)
    assert torch.equal(bare, h)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,I,E", SIZES)
def test_hidden_kept_in_8_bits(R, K, I, E, dtype):
    t = DTYPES[dtype]
    nb = -(-I // 32)
    x, w = randn(1, R, K, dtype=t), randn(2, E, 2 * I, K, dtype=t, std=K ** -0.5)
    off = offsets_of(3, R, E, before=R > 200, behind=R > 60)
    h, bare = sevens(R, I, t), sevens(R, I, t)
    codes = torch.full((R, 2 * I), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((R, 2 * nb), 77, dtype=torch.uint8, device="cuda")
    moe.experts_hidden(x, off, w, h, codes=codes, scales=scales)
    moe.experts_hidden(x, off, w, bare)
    assert torch.equal(h, bare)
    _, rp = o.hidden(f64(x), off.tolist(), f64(w), "silu", np.zeros((R, I)), np.zeros((R, 2 * I)))
    sp = hidden_slack(rp, magnitude(x, off, w), K)[0]
    c, s = codes.cpu().numpy().astype(np.int64), scales.cpu().numpy().astype(np.int64)
    mine = np.zeros(R, bool)
    for _, a, b in o.segments(off.tolist(), R):
        mine[a:b] = True
    assert (c[~mine] == 99).all() and (s[~mine] == 77).all()
    for half in range(2):
        cc, ss, v, e = (m[mine][:, half * n:(half + 1) * n] for m, n in ((c, I), (s, nb), (rp, I), (sp, I)))
        step = 2.0 ** (ss[:, np.arange(I) // 32] - 133)
        assert (np.abs(cc * step - v) <= step / 2 + e).all()
        for b in range(nb):   # the least scale, for the values as far off as they may be
            at = slice(b * 32, (b + 1) * 32)
            for lo, sign in ((False, 1), (True, -1)):
                near = np.maximum(np.abs(v[:, at]) + sign * e[:, at], 0)
                want = o.encode(near)[1][:, 0]
                assert ((ss[:, b] >= want) if lo else (ss[:, b] <= want)).all()


@pytest.mark.parametrize("keep", ["type", "8 bits"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,H,I,E", SIZES)
def test_hidden_backward(R, H, I, E, dtype, keep, act="silu"):
    t = DTYPES[dtype]
    nb = -(-I // 32)
    d_out, w = randn(1, R, H, dtype=t), randn(2, E, H, I, dtype=t, std=H ** -0.5)
    off = offsets_of(3, R, E, before=R > 200, behind=R > 60)
    pre = randn(5, R, 2 * I, dtype=t, std=2.0)
    kept = dict(pre=pre)
    if keep == "8 bits":
        act = "gelu"
        codes, scales = torch.empty(R, 2 * I, dtype=torch.int8, device="cuda"), torch.empty(R, 2 * nb, dtype=torch.uint8, device="cuda")
        for i in (0, 1):
            moe.rows_encode(pre[:, i * I:(i + 1) * I], codes[:, i * I:(i + 1) * I], scales[:, i * nb:(i + 1) * nb])
        kept = dict(codes=codes, scales=scales)
        c, s = codes.cpu().numpy().astype(np.int64), scales.cpu().numpy().astype(np.int64)
        p = np.concatenate([o.decode(c[:, :I], s[:, :nb]), o.decode(c[:, I:], s[:, nb:])], 1)
    else:
        p = f64(pre)
    d_pre, h = sevens(R, 2 * I, t), sevens(R, I, t)
    moe.experts_hidden_backward(d_out, off, w, d_pre, hidden=h, activation=act, **kept)
    rp, rh, dh = o.hidden_backward(f64(d_out), off.tolist(), f64(w), p, act, np.full((R, 2 * I), 7.0), np.full((R, I), 7.0))
    e = (H + 1) * ULP * o.hidden_backward(np.abs(f64(d_out)), off.tolist(), np.abs(f64(w)), p, act, np.zeros((R, 2 * I)),
                                          np.zeros((R, I)))[2]
    g, u = np.abs(p[:, :I]), np.abs(p[:, I:])
    dh = np.abs(dh) + e
    # the slope is a sum of terms up to 1 + g^2 in size
    assert_near(d_pre, rp, t, np.concatenate([e * u * 1.13 + dh * u * 2.0 ** -20 * (1 + g * g), e * g + dh * g * 2.0 ** -20], 1))
    assert_near(h, rh, t, 2.0 ** -20 * g * u)
    alone = sevens(R, 2 * I, t)
    moe.experts_hidden_backward(d_out, off, w, alone, activation=act, **kept)
    assert torch.equal(alone, d_pre)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,M,E", [s for s in SIZES if s[0] < 1000])
def test_weight_gradient_from_8_bits(R, K, M, E, dtype):
    """The same bits as from the values read back."""
    t = DTYPES[dtype]
    x, w, off = randn(1, R, K, dtype=t), randn(2, E, M, K, dtype=t), offsets_of(3, R, E)
    d_out = randn(4, R, M, dtype=t)
    codes = torch.empty(R, K, dtype=torch.int8, device="cuda")
    scales = torch.empty(R, -(-K // 32), dtype=torch.uint8, device="cuda")
    moe.rows_encode(x, codes, scales)
    back = torch.empty_like(x)
    moe.rows_decode(codes, scales, back)
    a, b = torch.empty(E, M, K, device="cuda"), torch.empty(E, M, K, device="cuda")
    moe.experts_product_backward(d_out, off, w, codes=codes, scales=scales, d_w=a)
    moe.experts_product_backward(d_out, off, w, x=back, d_w=b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,C", [(1, 1), (1, 31), (3, 32), (5, 33), (70, 100), (9, 256), (130, 1001), (33, 2048), (2, 5000)])
def test_rows_in_8_bits(R, C, dtype):
    t = DTYPES[dtype]
    # sizes over the type's range, zeros, blocks of zeros, values next to a border
    g = torch.Generator().manual_seed(C)
    v = torch.randn(R, C, generator=g) * torch.exp2(torch.randint(-20, 12, (R, 1), generator=g).float())
    v[torch.rand(R, C, generator=g) < 0.1] = 0
    v[0] = torch.round(v[0] * 8) / 16
    if R > 4:
        v[3] = 0
        v[4, :32] = 0
    x = v.to(t).cuda()
    codes = torch.full((R, C), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((R, -(-C // 32)), 77, dtype=torch.uint8, device="cuda")
    moe.rows_encode(x, codes, scales)
    rc, rs = o.encode(f64(x))
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    for u in DTYPES.values():
        back = torch.full((R, C), 7.0, dtype=u, device="cuda")
        moe.rows_decode(codes, scales, back)
        assert torch.equal(back.cpu(), torch.from_numpy(o.decode(rc, rs, torch.finfo(u).max)).to(u))


def test_rows_in_8_bits_at_the_ends_of_the_types():
    """Largest, smallest and subnormal values, infinities and NaN, beside rows that hold none."""
    for t in DTYPES.values():
        f = torch.finfo(t)
        tiny = f.smallest_normal * f.eps
        x = torch.ones(6, 64, dtype=t)
        x[0, 3], x[0, 40] = f.max, -f.max
        x[1] = 0
        x[1, 5], x[1, 6], x[1, 50] = tiny, -3 * tiny, f.smallest_normal
        x[2, 7], x[3, 63] = float("inf"), float("nan")
        x[4, :32] = float("-inf")
        x = x.cuda()
        codes, scales = torch.empty(6, 64, dtype=torch.int8, device="cuda"), torch.empty(6, 2, dtype=torch.uint8, device="cuda")
        moe.rows_encode(x, codes, scales)
        rc, rs = o.encode(f64(x))
        assert np.array_equal(scales.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)
        assert rs[2].tolist() == [255, rs[5, 1]] and rs[3, 1] == 255 and rs[4, 0] == 255
        back = torch.empty_like(x)
        moe.rows_decode(codes, scales, back)
        ref = o.decode(rc, rs, f.max)
        assert np.array_equal(f64(back), torch.from_numpy(ref).to(t).double().numpy(), equal_nan=True)
        assert torch.isfinite(back[0]).all() and torch.isnan(back[2, :32]).all() and (back[2, 32:] == 1).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides(dtype):
    """Column ranges of wider matrices, at any element: the same bits as from contiguous ones."""
    t = DTYPES[dtype]
    R, K, I, E, nb = 300, 128, 96, 3, 3
    off = offsets_of(3, R, E, 1, 2)
    x, w, wd = randn(1, R, K, dtype=t), randn(2, E, 2 * I, K, dtype=t), randn(6, E, K, I, dtype=t)
    d = randn(4, R, K, dtype=t)

    def chain(at):
        """Every operator on matrices of row distances at(columns) and offsets."""
        m = lambda C, ty=t: sevens(R, C, ty, *at(C))  # noqa: E731
        q = torch.zeros(R, at(2 * I)[0] + 8, dtype=torch.int8, device="cuda")[:, at(1)[1]:at(1)[1] + 2 * I]
        s = torch.zeros(R, 2 * nb + at(1)[1], dtype=torch.uint8, device="cuda")[:, at(1)[1]:]
        xs, ds = place(x, *at(K)), place(d, *at(K))
        h, pre, h2, out, d_pre, d_x, back = m(I), m(2 * I), m(I), m(K), m(2 * I), m(K), m(I)
        dw, dwd = torch.empty(E, 2 * I, K, device="cuda"), torch.empty(E, K, I, device="cuda")
        moe.experts_hidden(xs, off, w, h, pre=pre)
        moe.experts_hidden(xs, off, w, h2, codes=q, scales=s)
        moe.rows_decode(q[:, :I], s[:, :nb], back)
        moe.experts_product(h, off, wd, out)
        moe.experts_hidden_backward(ds, off, wd, d_pre, hidden=h2, pre=pre)
        moe.experts_product_backward(d_pre, off, w, x=xs, d_x=d_x, d_w=dw)
        moe.experts_product_backward(ds, off, wd, x=h2, d_w=dwd)
        return [v.clone() for v in (h, pre, q, s, back, out, d_pre, h2, d_x, dw, dwd)]

    plain = chain(lambda C: (C, 0))
    for at in (lambda C: (C + 8, 0), lambda C: (C + 1, 1), lambda C: (C + 3, 5)):
        for a, b in zip(plain, chain(at)):
            assert torch.equal(a, b)


def test_weights_at_any_element():
    R, K, M, E = 80, 64, 64, 2
    off = offsets_of(1, R, E)
    x, w = randn(1, R, K, dtype=torch.bfloat16), randn(2, E, M, K, dtype=torch.bfloat16)
    odd = torch.empty(E * M * K + 3, dtype=torch.bfloat16, device="cuda")[3:].view(E, M, K).copy_(w)
    a, b, c, d = (torch.zeros(R, K, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    moe.experts_product(x, off, w, a)
    moe.experts_product(x, off, odd, b)
    moe.experts_product_backward(x, off, w, d_x=c)
    moe.experts_product_backward(x, off, odd, d_x=d)
    assert torch.equal(a, b) and torch.equal(c, d)


@pytest.mark.parametrize("offsets", [[-5, 10, 4, 1000], [0, 0, 0, 0], [40, 40, 40, 40], [50, 2, 30, 7], [2 ** 31 - 1, 0, 5, 6],
                                     [-2 ** 31, -1, 20, 2 ** 31 - 1]])
@pytest.mark.parametrize("R", [6, 40, 600])
def test_offsets_out_of_order_or_range(offsets, R):
    """An offset counts as at least those before it and as 0 .. R."""
    t, K, M, E = torch.bfloat16, 64, 96, 3
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    x, w, d_out = randn(1, R, K, dtype=t), randn(2, E, M, K, dtype=t), randn(4, R, M, dtype=t)
    out, d_x, d_w = sevens(R, M, t), sevens(R, K, t), torch.full((E, M, K), 7.0, device="cuda")
    moe.experts_product(x, off, w, out)
    moe.experts_product_backward(d_out, off, w, x=x, d_x=d_x, d_w=d_w)
    assert_near(out, o.product(f64(x), offsets, f64(w), np.full((R, M), 7.0)), t, 65 * ULP * magnitude_at(x, offsets, w))
    rx, rw = o.product_backward(f64(d_out), f64(x), offsets, f64(w), np.full((R, K), 7.0))
    mx, mw = o.product_backward(np.abs(f64(d_out)), np.abs(f64(x)), offsets, np.abs(f64(w)), np.zeros((R, K)))
    assert_near(d_x, rx, t, 97 * ULP * mx)
    assert_near(d_w, rw, torch.float32, (R + 17) * ULP * mw)


def magnitude_at(x, offsets, w):
    return o.product(np.abs(f64(x)), offsets, np.abs(f64(w)), np.zeros((x.shape[0], w.shape[1])))


@pytest.mark.parametrize("R", [5, 300])
def test_no_rows_value_enters_another_row(R):
    """Infinities and NaN in one row, and in rows of no expert."""
    t, K, I, E = torch.float16, 80, 64, 2
    off = torch.tensor([1, 3, R - 1], dtype=torch.int32).cuda()
    x, w, wd = randn(1, R, K, dtype=t), randn(2, E, 2 * I, K, dtype=t), randn(5, E, K, I, dtype=t)
    h, out = sevens(R, I, t), sevens(R, K, t)
    moe.experts_hidden(x, off, w, h)
    moe.experts_product(h, off, wd, out)
    y = x.clone()
    y[0], y[R - 1], y[2, 3], y[3, 5] = float("nan"), float("inf"), float("inf"), float("nan")
    h2, out2 = sevens(R, I, t), sevens(R, K, t)
    moe.experts_hidden(y, off, w, h2)
    moe.experts_product(h2, off, wd, out2)
    same = [i for i in range(R) if i not in (2, 3)]
    assert torch.equal(h[same], h2[same]) and torch.equal(out[same], out2[same])
    assert not torch.isfinite(out2[2]).all() and torch.isnan(out2[3]).all()
    # and in the gradients: rows of no expert are not read, however they look
    d_w, d_w2, d_x = torch.empty(E, 2 * I, K, device="cuda"), torch.empty(E, 2 * I, K, device="cuda"), sevens(R, K, t)
    d = randn(7, R, 2 * I, dtype=t)
    moe.experts_product_backward(d, off, w, x=x, d_w=d_w)
    z, e = x.clone(), d.clone()
    z[0], z[R - 1], e[0], e[R - 1] = float("nan"), float("inf"), float("inf"), float("nan")
    moe.experts_product_backward(e, off, w, x=z, d_x=d_x, d_w=d_w2)
    assert torch.equal(d_w, d_w2) and (d_x[[0, R - 1]] == 7).all() and torch.isfinite(d_x).all()


def test_activations_at_large_arguments():
    """silu and gelu of large and infinite gates are 0 or the gate, and the slopes 0 or 1."""
    I = 32
    w = torch.eye(2 * I, dtype=torch.float32).reshape(1, 2 * I, 2 * I).cuda()
    x = torch.ones(1, 2 * I, device="cuda")
    big = torch.tensor([-1e30, -200.0, -89.0, -30.0, 30.0, 89.0, 200.0, 1e30], device="cuda")
    x[0, :8] = big
    off = torch.tensor([0, 1], dtype=torch.int32).cuda()
    for act in ("silu", "gelu"):
        h, pre = torch.empty(1, I, device="cuda"), torch.empty(1, 2 * I, device="cuda")
        moe.experts_hidden(x, off, w, h, activation=act, pre=pre)
        assert torch.equal(pre, x)
        assert (h[0, :3].abs() < 1e-30).all() and torch.equal(h[0, 4:8], big[4:])
        d_pre = torch.empty(1, 2 * I, device="cuda")
        moe.experts_hidden_backward(torch.ones(1, I, device="cuda"), off, torch.eye(I, device="cuda").reshape(1, I, I), d_pre,
                                    activation=act, pre=x)
        assert torch.equal(d_pre[0, 4:8], torch.ones(4, device="cuda")) and (d_pre[0, :3].abs() < 1e-30).all()


def test_empty_calls():
    t = torch.bfloat16
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    none, w = torch.empty(0, 16, dtype=t, device="cuda"), randn(1, 3, 16, 16, dtype=t)
    moe.experts_product(none, off, w, none.clone())
    moe.experts_hidden(none, off, w, torch.empty(0, 8, dtype=t, device="cuda"))
    d_w = torch.full((3, 16, 16), 7.0, device="cuda")
    moe.experts_product_backward(none, off, w, x=none, d_x=none.clone(), d_w=d_w)
    assert not d_w.any()
    moe.rows_encode(none, torch.empty(0, 16, dtype=torch.int8, device="cuda"), torch.empty(0, 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,M,E", [(700, 130, 100, 4), (2600, 64, 72, 1)])
def test_same_bits_again(R, K, M, E, dtype):
    t = DTYPES[dtype]
    x, w, d, off = randn(1, R, K, dtype=t), randn(2, E, M, K, dtype=t), randn(3, R, M, dtype=t), offsets_of(4, R, E)
    runs = []
    for _ in range(3):
        d_x, d_w = sevens(R, K, t), torch.empty(E, M, K, device="cuda")
        moe.experts_product_backward(d, off, w, x=x, d_x=d_x, d_w=d_w)
        runs.append((d_x, d_w))
    for d_x, d_w in runs[1:]:
        assert torch.equal(d_x, runs[0][0]) and torch.equal(d_w, runs[0][1])


def test_split_rows_joined():
    """One expert of many rows: its weights' gradient is made in runs of rows that are joined."""
    R, K, M = 9000, 96, 160
    assert moe.gpu_lib().moe_experts_product_workspace(R, K, M, 1) > 0
    off = torch.tensor([3, R - 5], dtype=torch.int32).cuda()
    for t in DTYPES.values():
        x, w, d = randn(1, R, K, dtype=t), randn(2, 1, M, K, dtype=t), randn(3, R, M, dtype=t)
        d_w = torch.empty(1, M, K, device="cuda")
        moe.experts_product_backward(d, off, w, x=x, d_w=d_w)
        a, b = f64(d)[3:R - 5], f64(x)[3:R - 5]
        # roundings of long sums are independent: 4 standard deviations of sqrt(R) of them, and cut ones R / 16 (a
        # matrix instruction adds 16 rows or more in 16-bit types; the fp32 one 2)
        size = np.abs(a).T @ np.abs(b)
        assert_near(d_w[0], a.T @ b, torch.float32, (R / (2 if t is torch.float32 else 16) + 20) * ULP * size)
