"""Experts' products at sizes of the larger tiles, and rows far apart in memory, against float64 (oracle/experts.py)."""
import numpy as np
import pytest
import torch

import expert_offload_lru_amd as moe
from oracle import experts as o
from test_gpu_experts import ULP, hidden_slack, magnitude, offsets_of, sevens
from token_harness import DTYPES, assert_near, f64, randn

pytestmark = pytest.mark.gpu

# 192 tiles of 256 x 256 and more, and fewer, with reductions of 1 to 9 steps; odd widths in tiles of 128 x 128
LARGE = [(6200, 96, 2048, 5), (16500, 40, 776, 3), (4096, 96, 2048, 5), (8200, 32, 1024, 3), (3900, 288, 2304, 1), (3840, 40, 2032, 2), (4100, 71, 1001, 6), (1000, 9, 4001, 2)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,M,E", LARGE)
def test_products(R, K, M, E, dtype):
    t = DTYPES[dtype]
    x, w, off, d = randn(1, R, K, dtype=t), randn(2, E, M, K, dtype=t), offsets_of(3, R, E, 1, 2), randn(4, R, M, dtype=t)
    out = sevens(R, M, t)
    moe.experts_product(x, off, w, out)
    assert_near(out, o.product(f64(x), off.tolist(), f64(w), np.full((R, M), 7.0)), t, (K + 1) * ULP * magnitude(x, off, w))
    # d_x with the widths exchanged: [R, M] of columns, from K
    v, d_x = randn(5, E, K, M, dtype=t), sevens(R, M, t)
    moe.experts_product_backward(x, off, v, d_x=d_x)
    ref, mag = (o.product_backward(a, np.zeros((R, M)), off.tolist(), b, c)[0] for a, b, c in (
        (f64(x), f64(v), np.full((R, M), 7.0)), (np.abs(f64(x)), np.abs(f64(v)), np.zeros((R, M)))))
    assert_near(d_x, ref, t, (K + 1) * ULP * mag)
    assert torch.equal(out[0], d_x[0])   # no expert's row


@pytest.mark.parametrize("keep", ["none", "type", "8 bits"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,I,E", [(6200, 64, 1024, 5), (12600, 104, 520, 2), (4096, 64, 1024, 5), (7900, 104, 520, 2), (4100, 71, 501, 6)])
def test_hidden(R, K, I, E, dtype, keep):
    t, nb = DTYPES[dtype], -(-I // 32)
    x, w, off = randn(1, R, K, dtype=t), randn(2, E, 2 * I, K, dtype=t, std=K ** -0.5), offsets_of(3, R, E, 1, 2)
    h, pre = sevens(R, I, t), sevens(R, 2 * I, t)
    codes, scales = torch.full((R, 2 * I), 99, dtype=torch.int8, device="cuda"), torch.full((R, 2 * nb), 77, dtype=torch.uint8, device="cuda")
    kept = dict(none={}, type=dict(pre=pre)).get(keep, dict(codes=codes, scales=scales))
    moe.experts_hidden(x, off, w, h, activation="gelu", **kept)
    rh, rp = o.hidden(f64(x), off.tolist(), f64(w), "gelu", np.full((R, I), 7.0), np.full((R, 2 * I), 7.0))
    sp, sh = hidden_slack(rp, magnitude(x, off, w), K)
    assert_near(h, rh, t, sh)
    if keep == "type":
        assert_near(pre, rp, t, sp)
    if keep == "8 bits":
        mine = slice(1, R - 2)
        for half in range(2):
            s = scales[mine, half * nb:(half + 1) * nb].cpu().numpy().astype(int)
            step = 2.0 ** (s[:, np.arange(I) // 32] - 133)
            at = slice(half * I, (half + 1) * I)
            got = codes[mine, at].cpu().numpy() * step
            assert (np.abs(got - rp[mine, at]) <= step / 2 + sp[mine, at]).all()
        assert (codes[[0, R - 1]] == 99).all() and (scales[[0, R - 1]] == 77).all()


@pytest.mark.parametrize("keep", ["type", "8 bits"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,H,I,E", [(6200, 64, 2048, 5), (12600, 104, 1032, 2), (4096, 64, 2048, 5), (7900, 104, 1032, 2), (4100, 71, 1001, 3)])
def test_hidden_backward(R, H, I, E, dtype, keep):
    t, nb = DTYPES[dtype], -(-I // 32)
    d_out, w, off = randn(1, R, H, dtype=t), randn(2, E, H, I, dtype=t, std=H ** -0.5), offsets_of(3, R, E, 1, 2)
    pre = randn(5, R, 2 * I, dtype=t, std=2.0)
    kept, p = dict(pre=pre), f64(pre)
    if keep == "8 bits":
        codes, scales = torch.empty(R, 2 * I, dtype=torch.int8, device="cuda"), torch.empty(R, 2 * nb, dtype=torch.uint8, device="cuda")
        back = torch.empty(R, 2 * I, device="cuda")
        for i in (0, 1):
            q, s = codes[:, i * I:(i + 1) * I], scales[:, i * nb:(i + 1) * nb]
            moe.rows_encode(pre[:, i * I:(i + 1) * I], q, s)
            moe.rows_decode(q, s, back[:, i * I:(i + 1) * I])
        kept, p = dict(codes=codes, scales=scales), f64(back)
    d_pre, h = sevens(R, 2 * I, t), sevens(R, I, t)
    moe.experts_hidden_backward(d_out, off, w, d_pre, hidden=h, **kept)
    rp, rh, dh = o.hidden_backward(f64(d_out), off.tolist(), f64(w), p, "silu", np.full((R, 2 * I), 7.0), np.full((R, I), 7.0))
    e = (H + 1) * ULP * magnitude_t(d_out, off, w)
    g, u, dh = np.abs(p[:, :I]), np.abs(p[:, I:]), np.abs(dh) + e
    assert_near(d_pre, rp, t, np.concatenate([e * u * 1.13 + dh * u * 2.0 ** -20 * (1 + g * g), e * g + dh * g * 2.0 ** -20], 1))
    assert_near(h, rh, t, 2.0 ** -20 * g * u)


def magnitude_t(d_out, off, w):
    return o.product_backward(np.abs(f64(d_out)), np.zeros((d_out.shape[0], w.shape[2])), off.tolist(), np.abs(f64(w)),
                              np.zeros((d_out.shape[0], w.shape[2])))[0]


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,M,N,E", [(17000, 520, 776, 130), (5000, 1024, 768, 3), (600, 1024, 2048, 4), (9000, 96, 160, 1), (2100, 203, 301, 2)])
def test_weight_gradients(R, M, N, E, dtype, codes):
    """Whole experts and runs of rows; values that add without a rounding, so that every row counts exactly."""
    t = DTYPES[dtype]
    g = torch.Generator().manual_seed(R)
    # small whole numbers: products and sums are whole numbers below 2^24
    x = torch.randint(-16, 17, (R, M), generator=g).to(t).cuda()
    d = torch.randint(-8, 9, (R, N), generator=g).to(t).cuda()
    off = offsets_of(3, R, E, 3, 4)
    d_w, w = torch.full((E, N, M), 7.0, device="cuda"), torch.empty(E, N, M, dtype=t, device="cuda")
    given = dict(x=x)
    if codes:
        q, s = torch.empty(R, M, dtype=torch.int8, device="cuda"), torch.empty(R, -(-M // 32), dtype=torch.uint8, device="cuda")
        moe.rows_encode(x, q, s)   # 16 is a power of two times a code: exact
        given = dict(codes=q, scales=s)
    moe.experts_product_backward(d, off, w, d_w=d_w, **given)
    xs, ds = x.double(), d.double()
    for e, a, b in o.segments(off.tolist(), R):
        assert torch.equal(d_w[e].double(), ds[a:b].T.contiguous() @ xs[a:b])


@pytest.mark.parametrize("ld", [4194240, 4194304 + 8, 4194304 * 2 + 1])
def test_rows_far_apart(ld):
    """Row distances next to what 31-bit offsets reach over 256 rows, and beyond: the same bits as from contiguous rows."""
    t, R, K, M, E = torch.bfloat16, 300, 64, 96, 2
    off = offsets_of(3, R, E, 1, 2)
    x, w, d = randn(1, R, K, dtype=t), randn(2, E, M, K, dtype=t), randn(4, R, M, dtype=t)
    buf = torch.empty(R * ld, dtype=t, device="cuda")
    far = lambda v: buf.view(R, ld)[:, :v.shape[1]].copy_(v)  # noqa: E731
    a, b, c, e = sevens(R, M, t), sevens(R, M, t), sevens(R, K, t), sevens(R, K, t)
    dw, dw2 = torch.empty(E, M, K, device="cuda"), torch.empty(E, M, K, device="cuda")
    moe.experts_product(x, off, w, a)
    moe.experts_product(far(x), off, w, b)
    assert torch.equal(a, b)
    moe.experts_product_backward(d, off, w, x=x, d_x=c, d_w=dw)
    moe.experts_product_backward(far(d), off, w, x=x, d_x=e, d_w=dw2)
    assert torch.equal(c, e) and torch.equal(dw, dw2)
    moe.experts_product_backward(d, off, w, x=far(x), d_w=dw2)
    assert torch.equal(dw, dw2)
    out = far(torch.full((R, M), 7.0, dtype=t, device="cuda"))
    moe.experts_product(x, off, w, out)
    assert torch.equal(a, out)
    # rows in 8 bits
    q, s = torch.empty(R, K, dtype=torch.int8, device="cuda"), torch.empty(R, 2, dtype=torch.uint8, device="cuda")
    moe.rows_encode(far(x), q, s)
    moe.experts_product_backward(d, off, w, codes=q, scales=s, d_w=dw)
    bytes_ = buf.view(torch.int8)
    q2 = bytes_[:2 * R * ld].view(R, 2 * ld)[:, :K].copy_(q)
    moe.experts_product_backward(d, off, w, codes=q2, scales=s, d_w=dw2)
    assert torch.equal(dw, dw2)
    back, near = far(x), torch.empty_like(x)
    moe.rows_decode(q, s, near)
    moe.rows_decode(q, s, back)
    assert torch.equal(near, back)


def test_many_experts():
    """1024 experts, 1 to 3 rows each and some none."""
    t, E, K, M = torch.float16, 1024, 40, 24
    counts = np.random.default_rng(1).integers(0, 4, E)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
    R = int(off[-1])
    x, w, d = randn(1, R, K, dtype=t), randn(2, E, M, K, dtype=t), randn(4, R, M, dtype=t)
    out, d_x, d_w = sevens(R, M, t), sevens(R, K, t), torch.full((E, M, K), 7.0, device="cuda")
    moe.experts_product(x, off, w, out)
    moe.experts_product_backward(d, off, w, x=x, d_x=d_x, d_w=d_w)
    assert_near(out, o.product(f64(x), off.tolist(), f64(w), np.zeros((R, M))), t, (K + 1) * ULP * magnitude(x, off, w))
    rx, rw = o.product_backward(f64(d), f64(x), off.tolist(), f64(w), np.zeros((R, K)))
    mx, mw = o.product_backward(np.abs(f64(d)), np.abs(f64(x)), off.tolist(), np.abs(f64(w)), np.zeros((R, K)))
    assert_near(d_x, rx, t, (M + 1) * ULP * mx)
    assert_near(d_w, rw, torch.float32, 8 * ULP * mw)


def whole(seed, *shape, dtype, most=8):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,M,E", [(40, 64, 1), (700, 2432, 2), (6200, 2048, 5)])
def test_every_number_of_steps(R, M, E, dtype):
    """Reductions of 1 to 20 steps and their remainders by the steps held at a time, in each tile; sums of whole numbers are exact,
    so a load that came late or a step too many shows in any bit."""
    t = DTYPES[dtype]
    off = offsets_of(3, R, E, 1, 2)
    piece = 16 // torch.empty((), dtype=t).element_size()
    lengths = [n * 4 * piece - cut for n in range(1, 20 if R < 1000 else 10) for cut in (0, piece)]
    for K in lengths:
        x, w = whole(K, R, K, dtype=t), whole(K + 1, E, M, K, dtype=t)
        v = w.transpose(1, 2).contiguous()
        out, d_x = sevens(R, M, t), sevens(R, M, t)
        moe.experts_product(x, off, w, out)
        moe.experts_product_backward(x, off, v, d_x=d_x)
        want = torch.full((R, M), 7.0, dtype=t, device="cuda")
        for e, a, b in o.segments(off.tolist(), R):
            want[a:b] = (x[a:b].float() @ v[e].float()).to(t)   # exact in fp32
        assert torch.equal(out, want) and torch.equal(d_x, want), K


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,E", [(64, 72, 1), (1024, 768, 3)])
def test_weight_gradients_of_every_number_of_steps(M, N, E, dtype):
    t = DTYPES[dtype]
    for rows in [*range(1, 7), *range(15, 330, 21), *((1100, 1130, 1160, 1190) if E > 1 else ())]:
        R = E * rows
        off = torch.arange(0, R + 1, rows, dtype=torch.int32).cuda()
        x, d, w = whole(rows, R, M, dtype=t), whole(rows + 1, R, N, dtype=t), torch.empty(E, N, M, dtype=t, device="cuda")
        q, s = torch.empty(R, M, dtype=torch.int8, device="cuda"), torch.empty(R, M // 32, dtype=torch.uint8, device="cuda")
        moe.rows_encode(x, q, s)
        a, b = torch.empty(E, N, M, device="cuda"), torch.empty(E, N, M, device="cuda")
        moe.experts_product_backward(d, off, w, x=x, d_w=a)
        moe.experts_product_backward(d, off, w, codes=q, scales=s, d_w=b)
        want = torch.stack([d[i * rows:(i + 1) * rows].double().T.contiguous() @ x[i * rows:(i + 1) * rows].double() for i in range(E)])
        assert torch.equal(a.double(), want) and torch.equal(b, a), rows
