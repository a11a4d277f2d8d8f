"""Low-rank adapters and their gradients (include/moe_tokens.h) against the float64 oracle."""
import numpy as np
import pytest
import torch

import expert_offload_lru_amd as moe
import synth
from gpu_harness import Model
from oracle import tokens as ref
from token_harness import DTYPES, assert_near, assert_norm, f64, order_buffers, place, randn

pytestmark = pytest.mark.gpu

# T, n, r, inner, outer, dtype, wtype, order of the rows' adapters
SHAPES = [
    (1, 1, 1, 1, 1, "f32", "f32", "mixed"),
    (1, 4, 16, 2048, 2048, "bf16", "bf16", "mixed"),
    (1, 4, 8, 768, 2048, "f32", "bf16", "mixed"),
    (2, 3, 5, 7, 3, "f16", "f16", "mixed"),
    (9, 5, 3, 100, 70, "bf16", "bf16", "mixed"),
    (32, 40, 16, 512, 640, "f32", "f16", "mixed"),
    (33, 2, 64, 1000, 520, "f16", "f16", "mixed"),
    (100, 7, 12, 130, 1030, "bf16", "bf16", "mixed"),
    (300, 3, 8, 768, 256, "f32", "f32", "runs"),
    (600, 2, 16, 256, 2048, "bf16", "bf16", "runs"),
    (700, 9, 32, 520, 264, "f16", "f16", "runs"),
    (513, 3, 256, 192, 136, "bf16", "bf16", "runs"),
    (520, 2, 200, 72, 90, "f32", "bf16", "runs"),
    (1100, 40, 7, 66, 65, "bf16", "bf16", "runs"),
    (1025, 5, 33, 260, 129, "f32", "f32", "mixed"),
    (2050, 1, 128, 64, 64, "f16", "f16", "runs"),
    (640, 1000, 4, 40, 48, "bf16", "bf16", "mixed"),
    # many rows: blocks of 16 and 32, second adapters of a block done elsewhere, several pieces an adapter
    (4200, 9, 16, 64, 72, "bf16", "bf16", "runs"),
    (4500, 70, 24, 72, 64, "f16", "f16", "mixed"),
    (5000, 3, 48, 64, 64, "f32", "bf16", "runs"),
    (4100, 5, 100, 64, 136, "bf16", "bf16", "mixed"),
    (4111, 300, 32, 65, 64, "bf16", "bf16", "mixed"),
    (16500, 3, 24, 64, 64, "bf16", "bf16", "runs"),
    (33000, 5, 4, 24, 16, "bf16", "bf16", "mixed"),
    (9000, 270, 64, 64, 16, "f16", "f16", "runs"),
    # blocks of few rows, ranks dealt to workgroups
    (40, 3, 256, 2048, 2048, "bf16", "bf16", "mixed"),
    (20, 2, 200, 5000, 4000, "f16", "f16", "mixed"),
    (1, 2, 256, 70000, 65536, "bf16", "bf16", "mixed"),
    (150, 4, 64, 2048, 3000, "f32", "bf16", "runs"),
    # odd sizes copied to aligned rows
    (8200, 3, 5, 33, 17, "bf16", "bf16", "runs"),
    (8300, 4, 12, 100, 72, "f32", "f16", "mixed"),
    (9000, 2, 8, 72, 35, "f16", "f16", "runs"),
]


def which(seed, T, n, order):
    rng = np.random.default_rng(seed)
    if order == "mixed":
        return rng.integers(-1, n, T).astype(np.int32)
    at = np.searchsorted(np.sort(rng.integers(0, T + 1, n)), np.arange(T), side="right")
    return np.where(at == n, -1, at).astype(np.int32)


def make(T, n, r, inner, outer, dt, wt, order, seed=0):
    d, w = DTYPES[dt], DTYPES[wt]
    s = dict(adapter=torch.from_numpy(which(seed, T, n, order)).cuda(), x=randn(seed + 1, T, inner, dtype=d),
             a=randn(seed + 2, n, r, inner, dtype=w, std=inner ** -0.5), b=randn(seed + 3, n, outer, r, dtype=w, std=r ** -0.5),
             scale=randn(seed + 4, n), base=randn(seed + 5, T, outer, dtype=d), d_out=randn(seed + 6, T, outer, dtype=d),
             dx_base=randn(seed + 7, T, inner, dtype=d))
    return s


def numbers(s):
    return {k: (v.cpu().numpy() if k == "adapter" else f64(v)) for k, v in s.items()}


def sizes(m):
    return {k: (v if k == "adapter" else np.abs(v)) for k, v in m.items()}


def forward(s, base=None, out=None):
    if out is None:
        out = torch.full((s["x"].shape[0], s["b"].shape[1]), 9.0, dtype=s["x"].dtype, device="cuda")
    moe.adapters_forward(s["x"], s["adapter"], s["a"], s["b"], s["scale"], out, base=base)
    return out


# v and u are rounded to two parts of 8 bits or more before the second product of 16-bit types
SPLIT = {torch.float32: 0.0, torch.float16: 2.0 ** -16, torch.bfloat16: 2.0 ** -16}


def forward_slack(m, dtype, base):
    z = sizes(m)
    terms = z["a"].shape[2] + z["a"].shape[1] + 16
    size = ref.adapters(z["x"], m["adapter"], z["a"], z["b"], z["scale"])
    return (terms * 2.0 ** -23 + SPLIT[dtype]) * size + (2.0 ** -24 * np.abs(m["base"]) if base else 0)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_forward(shape):
    s = make(*shape, seed=100)
    m, dtype = numbers(s), s["x"].dtype
    terms = shape[3] + shape[2]
    plain = forward(s)
    want = ref.adapters(m["x"], m["adapter"], m["a"], m["b"], m["scale"])
    assert_near(plain, want, dtype, forward_slack(m, dtype, False))
    assert_norm(plain, want, dtype, terms, SPLIT[dtype])
    added = forward(s, base=s["base"])
    want = ref.adapters(m["x"], m["adapter"], m["a"], m["b"], m["scale"], m["base"])
    assert_near(added, want, dtype, forward_slack(m, dtype, True))
    none = torch.from_numpy((m["adapter"] < 0)).cuda()
    assert torch.equal(added[none], s["base"][none]) and not plain[none].any()
    same = s["base"].clone()
    assert torch.equal(forward(s, base=same, out=same), added)


def backward(s, dx_base=None, d_x=None, workspace=None):
    n, r, inner = s["a"].shape
    if d_x is None:
        d_x = torch.full(s["x"].shape, 9.0, dtype=s["x"].dtype, device="cuda")
    d_a, d_b = torch.full(s["a"].shape, 9.0, device="cuda"), torch.full(s["b"].shape, 9.0, device="cuda")
    moe.adapters_backward(s["d_out"], s["x"], s["adapter"], s["a"], s["b"], s["scale"], d_x, d_a, d_b, dx_base=dx_base,
                          workspace=workspace)
    return d_x, d_a, d_b


def check_backward(s, m, got, base):
    dtype, z = s["x"].dtype, sizes(m)
    T, (n, r, inner), outer = s["x"].shape[0], s["a"].shape, s["b"].shape[1]
    want = ref.adapters_backward(m["d_out"], m["x"], m["adapter"], m["a"], m["b"], m["scale"], m["dx_base"] if base else None)
    size = ref.adapters_backward(z["d_out"], z["x"], m["adapter"], z["a"], z["b"], z["scale"])
    slack = [((outer + r + 16) * 2.0 ** -23 + SPLIT[dtype]) * size[0] + (2.0 ** -24 * z["dx_base"] if base else 0),
             ((outer + T + 16) * 2.0 ** -23 + SPLIT[dtype]) * size[1], ((inner + T + 16) * 2.0 ** -23 + SPLIT[dtype]) * size[2]]
    for g, w, e, t in zip(got, want, slack, (dtype, torch.float32, torch.float32)):
        assert_near(g, w, t, e)
        assert_norm(g, w, t, inner + outer + T, SPLIT[dtype])


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_backward(shape):
    s = make(*shape, seed=200)
    m = numbers(s)
    got = backward(s)
    check_backward(s, m, got, False)
    added = backward(s, dx_base=s["dx_base"])
    check_backward(s, m, added, True)
    assert torch.equal(got[1], added[1]) and torch.equal(got[2], added[2])
    same = s["dx_base"].clone()
    assert torch.equal(backward(s, dx_base=same, d_x=same)[0], added[0])


@pytest.mark.parametrize("dt,wt", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("T", [19, 777])
def test_strides(dt, wt, T):
    s = make(T, 3, 10, 90, 75, dt, wt, "mixed", seed=300)
    want, wantb = forward(s, base=s["base"]), backward(s, dx_base=s["dx_base"])
    for ld, offset in ((91, 1), (96, 3)):
        t = dict(s, **{k: place(s[k], ld, offset) for k in ("x", "base", "d_out", "dx_base")})
        out, d_x = place(torch.zeros_like(s["base"]), ld, offset), place(torch.zeros_like(s["x"]), ld, offset)
        forward(t, base=t["base"], out=out)
        got = backward(t, dx_base=t["dx_base"], d_x=d_x)
        assert torch.equal(out, want)
        for g, w in zip(got, wantb):
            assert torch.equal(g, w)
        for v, cols in ((out, 75), (d_x, 90)):
            buf = v._base.clone()
            buf[offset:offset + T * ld].view(T, ld)[:, :cols] = 7.0
            assert (buf == 7.0).all()      # nothing written beside the rows


@pytest.mark.parametrize("T", [5, 900])
def test_ids_out_of_range_and_no_adapter_at_all(T):
    s = make(T, 3, 8, 64, 48, "bf16", "bf16", "mixed", seed=400)
    s["adapter"][0::3] = 3
    s["adapter"][1::3] = -2 ** 31
    m = numbers(s)
    assert_near(forward(s, base=s["base"]), ref.adapters(m["x"], m["adapter"], m["a"], m["b"], m["scale"], m["base"]),
                torch.bfloat16, forward_slack(m, torch.bfloat16, True))
    check_backward(s, m, backward(s), False)
    s["adapter"].fill_(2 ** 31 - 1)
    assert torch.equal(forward(s, base=s["base"]), s["base"]) and not forward(s).any()
    d_x, d_a, d_b = backward(s)
    assert not d_x.any() and not d_a.any() and not d_b.any()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [24, 1200])
def test_non_finite_values_stay_with_their_rows_and_adapters(dt, T):
    """Adapters beside each other in a block of rows: one's infinities and NaN reach its own rows only."""
    s = make(T, 4, 16, 128, 96, dt, dt, "mixed", seed=500)
    clean, cleanb = forward(s, base=s["base"]), backward(s)
    bad = s["adapter"] == 1
    s["a"][1, 3] = float("inf")
    s["b"][1, 5] = float("nan")
    s["x"][int(torch.nonzero(s["adapter"] == 2)[0, 0])] = float("nan")
    bad[int(torch.nonzero(s["adapter"] == 2)[0, 0])] = True
    out, (d_x, d_a, d_b) = forward(s, base=s["base"]), backward(s)
    assert torch.equal(out[~bad], clean[~bad])
    assert torch.isnan(out[s["adapter"] == 1][:, 5]).all()
    keep = s["adapter"] != 1
    assert torch.equal(d_x[keep], cleanb[0][keep])
    for g, c in ((d_a, cleanb[1]), (d_b, cleanb[2])):
        assert torch.equal(g[0], c[0]) and torch.equal(g[3], c[3])
    assert torch.isnan(d_a[2]).any()


def test_large_intermediate_values_in_fp16():
    """A x beyond fp16's range is held in fp32: only the result is rounded."""
    T, inner, outer, r = 40, 256, 64, 8
    s = make(T, 1, r, inner, outer, "f16", "f16", "mixed", seed=600)
    s["adapter"].zero_()
    s["x"].fill_(100.0)
    s["a"].fill_(20.0)                        # v = 512000
    s["b"].fill_(2.0 ** -12)
    for t in (1, T):
        u = dict(s, x=s["x"][:t], adapter=s["adapter"][:t], base=s["base"][:t])
        u["scale"] = torch.ones(1, device="cuda")
        assert torch.equal(forward(u), torch.full((t, outer), 1000.0, dtype=torch.float16, device="cuda"))
    many = dict(s, x=s["x"].repeat(30, 1), adapter=s["adapter"].repeat(30), scale=torch.ones(1, device="cuda"))
    assert (forward(many) == 1000.0).all()


@pytest.mark.parametrize("dt,wt", [("bf16", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("inner,outer,r", [(96, 72, 12), (96, 75, 8), (90, 72, 12)])
@pytest.mark.parametrize("T", [1300, 8300])
def test_strided_rows_with_and_without_room_for_copies(T, dt, wt, inner, outer, r):
    """Rows that no 16-byte piece fits: copied first where the workspace has room for it, else read as they lie."""
    n, lib = 4, moe.gpu_lib()
    s = make(T, n, r, inner, outer, dt, wt, "runs", seed=350)
    m, dtype = numbers(s), s["x"].dtype
    for ld_x, ld_out, offset in ((inner + 11, outer + 8, 0), (inner + 8, outer + 8, 1)):
        t = dict(s, **{k: place(s[k], ld, offset) for k, ld in (("x", ld_x), ("dx_base", ld_x), ("base", ld_out), ("d_out", ld_out))})
        want = ref.adapters(m["x"], m["adapter"], m["a"], m["b"], m["scale"], m["base"])
        for name in ("", "_strided"):
            bytes_f = getattr(lib, "moe_adapters_forward_workspace" + name)(T, inner, outer, n, r)
            bytes_b = getattr(lib, "moe_adapters_workspace" + name)(T, inner, outer, n, r)
            ws = torch.full((max(bytes_f, bytes_b) + 512,), 0xFF, dtype=torch.uint8, device="cuda")
            out, d_x = place(torch.zeros_like(s["base"]), ld_out, offset), place(torch.zeros_like(s["x"]), ld_x, offset)
            moe.adapters_forward(t["x"], s["adapter"], s["a"], s["b"], s["scale"], out, base=t["base"], workspace=ws[:bytes_f])
            assert (ws[bytes_f:] == 0xFF).all()
            assert_near(out, want, dtype, forward_slack(m, dtype, True))
            ws.fill_(0xFF)
            check_backward(s, m, backward(t, dx_base=t["dx_base"], d_x=d_x, workspace=ws[:bytes_b]), True)
            assert (ws[bytes_b:] == 0xFF).all()
            for v, ld, cols in ((out, ld_out, outer), (d_x, ld_x, inner)):
                buf = v._base.clone()
                buf[offset:offset + T * ld].view(T, ld)[:, :cols] = 7.0
                assert (buf == 7.0).all()


def test_millions_of_rows_a_workgroup_each():
    """A workgroup a row for unaligned rows without room for copies: the grid stays within a launch's limits."""
    T, n, r, inner, outer = (1 << 22) + 3, 3, 40, 8, 8
    g = torch.Generator(device="cuda").manual_seed(360)
    x = torch.randn(T, inner + 1, generator=g, device="cuda").bfloat16()[:, 1:]
    adapter = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32, device="cuda")
    a, b = randn(361, n, r, inner, dtype=torch.bfloat16), randn(362, n, outer, r, dtype=torch.bfloat16)
    scale, out = randn(363, n), torch.empty(T, outer, dtype=torch.bfloat16, device="cuda")
    need = moe.gpu_lib().moe_adapters_forward_workspace(T, inner, outer, n, r)
    moe.adapters_forward(x, adapter, a, b, scale, out, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    for part in (slice(0, 7), slice(T // 2, T // 2 + 9), slice(T - 9, T)):
        few = torch.empty_like(out[part])
        moe.adapters_forward(x[part], adapter[part].contiguous(), a, b, scale, few)
        assert torch.equal(out[part], few)


def test_no_rows():
    s = make(0, 3, 4, 10, 12, "f32", "f32", "mixed", seed=700)
    assert forward(s).shape == (0, 12)
    d_x, d_a, d_b = backward(s)
    assert not d_a.any() and not d_b.any()


def test_repeats_streams_and_a_kept_workspace_are_bitwise_equal():
    s = make(900, 5, 16, 256, 320, "bf16", "bf16", "runs", seed=800)
    out, grads = forward(s), backward(s)
    n = moe.gpu_lib().moe_adapters_workspace(900, 256, 320, 5, 16)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(st):
            assert torch.equal(forward(s), out)
            for g, w in zip(backward(s, workspace=ws), grads):
                assert torch.equal(g, w)


def test_two_calls_at_once():
    """Calls on two streams with tensors and workspaces of their own, in flight together."""
    sets = [make(1400, 6, 24, 256, 320, "bf16", "bf16", "runs", seed=820 + i) for i in range(2)]
    want = [(forward(s, base=s["base"]), *backward(s)) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for s, st, g in zip(sets, streams, got):
            with torch.cuda.stream(st):
                g.append((forward(s, base=s["base"]), *backward(s)))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for outputs in g:
            assert all(torch.equal(a, b) for a, b in zip(outputs, w))


def test_gradients_against_differences():
    """out is linear in x, in a and in b: a difference over a step of one is the derivative."""
    s = make(50, 3, 6, 40, 30, "f32", "f32", "mixed", seed=900)
    w = s["d_out"]
    grads = dict(zip(("x", "a", "b"), backward(s)))
    m = sizes(numbers(s))

    for name, g in grads.items():
        d = randn(910, *g.shape, std=float(s[name].std()))

        def loss(sign):
            return (forward(dict(s, **{name: s[name] + sign * d})).double() * w.double()).sum().item()

        z = dict(m, **{name: m[name] + np.abs(f64(d))})
        size = float((ref.adapters(z["x"], m["adapter"], z["a"], z["b"], z["scale"]) * z["d_out"]).sum())
        tol = 4 * (40 + 30 + 6 + 50) * 2.0 ** -24 * size
        assert abs((loss(1) - loss(-1)) / 2 - (g.double() * d.double()).sum().item()) < tol, name


def test_refusals():
    s = make(6, 2, 4, 16, 24, "bf16", "bf16", "mixed", seed=1000)
    out = torch.empty(6, 24, dtype=torch.bfloat16, device="cuda")

    def refused(code=moe.ERR_INVALID, out=out, **kw):
        t = dict(s, **kw)
        with pytest.raises(moe.MoeError) as e:
            moe.adapters_forward(t["x"], t["adapter"], t["a"], t["b"], t["scale"], out)
        assert e.value.code == code

    refused(a=s["a"].float(), b=s["b"].float())               # another type beside 16-bit activations
    refused(b=s["b"].half())
    refused(a=s["a"][:, :3])
    refused(a=s["a"][:, :, :15].contiguous())
    refused(adapter=s["adapter"].long())
    refused(adapter=s["adapter"][:-1])
    refused(scale=s["scale"].double())
    refused(x=s["x"].cpu())
    refused(x=s["x"][0])
    refused(out=out[:, :20])
    refused(out=torch.empty(24, 6, dtype=torch.bfloat16, device="cuda").t())
    refused(code=moe.ERR_UNSUPPORTED, x=s["x"][:1].expand(2 ** 32 + 6, 16))   # a size that 32 bits would cut to 6
    wide = torch.empty(6, 40, dtype=torch.bfloat16, device="cuda")
    refused(out=wide[:, :24], x=wide[:, 24:])                   # rows that interleave count as overlapping
    refused(code=moe.ERR_UNSUPPORTED, a=torch.zeros(2, 257, 16, dtype=torch.bfloat16, device="cuda"),
            b=torch.zeros(2, 24, 257, dtype=torch.bfloat16, device="cuda"))
    d_a, d_b, d_x = torch.empty(2, 4, 16, device="cuda"), torch.empty(2, 24, 4, device="cuda"), torch.empty_like(s["x"])

    def refused_back(code=moe.ERR_INVALID, d_a=d_a, d_b=d_b, d_x=d_x, workspace=None):
        with pytest.raises(moe.MoeError) as e:
            moe.adapters_backward(s["d_out"], s["x"], s["adapter"], s["a"], s["b"], s["scale"], d_x, d_a, d_b,
                                  workspace=workspace)
        assert e.value.code == code

    refused_back(d_a=d_a.bfloat16())
    refused_back(d_b=d_b[:1])
    refused_back(d_x=s["x"])
    refused_back(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    n = moe.gpu_lib().moe_adapters_workspace(6, 16, 24, 2, 4)
    refused_back(workspace=torch.empty(n + 16, dtype=torch.uint8, device="cuda")[4:])


# ------------------------------------------------------------------------- the operators together

class Chain:
    """A training step of per-expert adapters on the routed rows: dispatch, adapters, combine on top of the
    layer's output, and back."""

    def __init__(self, x, ids, gate, base, a, b, scale, d_out):
        self.x, self.ids, self.gate, self.base = x, ids, gate, base
        self.a, self.b, self.scale, self.d_out = a, b, scale, d_out
        T, k = ids.shape
        n, H, O = T * k, x.shape[1], b.shape[1]
        z = dict(dtype=x.dtype, device="cuda")
        self.o = order_buffers(T, k, a.shape[0])
        self.rows, self.prod, self.out = torch.zeros(n, H, **z), torch.zeros(n, O, **z), torch.empty(T, O, **z)
        self.d_prod, self.d_rows, self.d_x = torch.zeros(n, O, **z), torch.empty(n, H, **z), torch.empty(T, H, **z)
        self.d_gate, self.d_a, self.d_b = (torch.empty(v.shape, device="cuda") for v in (gate, a, b))
        need = moe.gpu_lib().moe_adapters_workspace(n, H, O, a.shape[0], a.shape[1])
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(self):
        o = self.o
        moe.tokens_dispatch(self.x, self.ids, self.a.shape[0], self.rows, **o)
        moe.adapters_forward(self.rows, o["expert"], self.a, self.b, self.scale, self.prod)
        moe.tokens_combine(self.prod, o["pos"], self.gate, self.out, base=self.base)
        moe.tokens_combine_backward(self.d_out, self.prod, o["pos"], self.gate, self.d_prod, self.d_gate)
        moe.adapters_backward(self.d_prod, self.rows, o["expert"], self.a, self.b, self.scale, self.d_rows, self.d_a,
                              self.d_b, workspace=self.ws)
        moe.tokens_dispatch_backward(self.d_rows, o["pos"], self.d_x)

    def results(self):
        return [v.clone() for v in (self.out, self.d_gate, self.d_x, self.d_a, self.d_b)]


def chain_reference(c, base):
    """The same step in float64, token by token."""
    x, gate, a, b, s, dy = (f64(v) for v in (c.x, c.gate, c.a, c.b, c.scale, c.d_out))
    ids = c.ids.cpu().numpy()
    out, d_gate, d_x, d_a, d_b = base.copy(), np.zeros(gate.shape), np.zeros(x.shape), np.zeros(a.shape), np.zeros(b.shape)
    for t in range(ids.shape[0]):
        for j, e in enumerate(ids[t]):
            if e < 0:
                continue
            v = a[e] @ x[t]
            y = s[e] * (b[e] @ v)
            out[t] += gate[t, j] * y
            d_gate[t, j] = dy[t] @ y
            u = s[e] * gate[t, j] * (b[e].T @ dy[t])
            d_x[t] += a[e].T @ u
            d_a[e] += np.outer(u, x[t])
            d_b[e] += s[e] * gate[t, j] * np.outer(dy[t], v)
    return out, d_gate, d_x, d_a, d_b


@pytest.mark.parametrize("b", [1, 12, 80])
def test_adapters_beside_the_layers_experts(b):
    """The layer's own routing and output, decode and prefill: its experts' adapters on top of it."""
    E, k, H, r = 16, 2, 256, 8
    m = Model(E, 8, k, H, 256, moe.Q_INT4_G32_F16, 1, seed=71)
    try:
        x = torch.from_numpy(synth.ar1_streams(72, b, 1, H)[0]).cuda()
        base = torch.empty_like(x)
        m.cache.forward(0, x, b, m.router[0], base, residual=True)
        torch.cuda.synchronize()
        ids, gate = m.cache.last_routing(b)
        c = Chain(x, torch.from_numpy(ids).cuda(), torch.from_numpy(gate).cuda(), base,
                  randn(73, E, r, H, dtype=torch.bfloat16, std=H ** -0.5), randn(74, E, H, r, dtype=torch.bfloat16, std=r ** -0.5),
                  randn(75, E), randn(76, b, H))
        c.step()
        for got, want in zip(c.results(), chain_reference(c, f64(base))):
            assert_norm(got, want, torch.float32, 4 * H + b)
    finally:
        m.close()


@pytest.mark.parametrize("T", [3, 400])
def test_captured_step(T):
    """The step captured into a graph, replayed with eager work and synchronizations between, new inputs in the
    same places: every replay equals the eager step."""
    E, k, H, r, O = 12, 3, 192, 16, 136
    ids = torch.from_numpy(np.random.default_rng(81).integers(-1, E, (T, k)).astype(np.int32)).cuda()
    c = Chain(randn(82, T, H, dtype=torch.bfloat16), ids, randn(83, T, k), randn(84, T, O, dtype=torch.bfloat16),
              randn(85, E, r, H, dtype=torch.bfloat16, std=H ** -0.5), randn(86, E, O, r, dtype=torch.bfloat16, std=0.25),
              randn(87, E), randn(88, T, O, dtype=torch.bfloat16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.step()
    for i in range(4):
        c.x.copy_(randn(90 + i, T, H, dtype=torch.bfloat16))
        c.ids.copy_(torch.from_numpy(np.random.default_rng(95 + i).integers(-1, E, (T, k)).astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        got = c.results()
        c.step()
        torch.cuda.synchronize()
        for g, w in zip(got, c.results()):
            assert torch.equal(g, w)
