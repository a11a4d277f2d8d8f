"""The operators together, as a training step and a decode step use them: norms around a block of routed experts,
what the backward pass needs kept in 8 bits; eagerly, captured, on other streams, beside torch's autograd."""
import numpy as np
import pytest
import torch

import expert_offload_lru_amd as moe
from oracle import experts as o
from oracle import tokens as ot
from token_harness import DTYPES, f64, order_buffers, picks, randn

pytestmark = pytest.mark.gpu
T, k, E, H, I = 90, 2, 5, 96, 72
PARAMS = ("w_post", "gate", "alpha", "w_pre")


def tensors(dtype, keep, seed=0, T=T):
    t, R, nb = DTYPES[dtype], T * k, -(-I // 32)
    z = lambda *s, ty=t: torch.zeros(s, dtype=ty, device="cuda")  # noqa: E731
    f = lambda *s: z(*s, ty=torch.float32)  # noqa: E731
    s = dict(x=randn(seed + 1, T, H, dtype=t), w=randn(seed + 2, E, 2 * I, H, dtype=t, std=H ** -0.5),
             wd=randn(seed + 3, E, H, I, dtype=t, std=I ** -0.5), mix=torch.softmax(randn(seed + 4, T, k), -1),
             w_pre0=randn(seed + 5, H) * 0.1 + 1, w_post=randn(seed + 6, H) * 0.1 + 1, alpha=randn(seed + 7, H) * 0.1 + 1,
             w_pre=randn(seed + 8, H) * 0.1 + 1, gate=randn(seed + 9, 3, H), ids=torch.from_numpy(picks(seed, T, k, E, 0.1)).cuda(),
             d_next=randn(seed + 10, T, H, dtype=t), d_res=randn(seed + 11, T, H, dtype=t))
    s.update(order_buffers(T, k, E), n0=z(T, H), st0=f(T, 2), rows=z(R, H), hid=z(R, I), out_rows=z(R, H), y=z(T, H), res=z(T, H),
             nxt=z(T, H), st=f(T, 2), d_x=z(T, H), d_y=z(T, H), d_rows=z(R, H), d_mix=f(T, k), d_pre=z(R, 2 * I), hid2=z(R, I),
             d_wd=f(E, H, I), d_xr=z(R, H), d_w=f(E, 2 * I, H), d_n0=z(T, H), d_total=z(T, H),
             d_w_pre0=f(H), **{"d_" + n: torch.zeros_like(s[n]) for n in PARAMS})
    s["per"] = -(-T // 3)
    if keep == "8 bits":
        i8, u8 = torch.int8, torch.uint8
        s.update(codes=z(R, 2 * I, ty=i8), scales=z(R, 2 * nb, ty=u8), xc=z(R, H, ty=i8), xs=z(R, -(-H // 32), ty=u8))
    else:
        s["pre"] = z(R, 2 * I)
    return s


def forward(s, stream=None):
    kw = dict(stream=stream)
    moe.block_norm(s["x"], None, None, w_pre=s["w_pre0"], normed=s["n0"], stats=s["st0"], **kw)
    moe.tokens_dispatch(s["n0"], s["ids"], E, s["rows"], s["offsets"], s["pos"], s["src"], s["expert"], **kw)
    if "codes" in s:
        moe.rows_encode(s["rows"], s["xc"], s["xs"], **kw)
    moe.experts_hidden(s["rows"], s["offsets"], s["w"], s["hid"], pre=s.get("pre"), codes=s.get("codes"), scales=s.get("scales"), **kw)
    moe.experts_product(s["hid"], s["offsets"], s["wd"], s["out_rows"], **kw)
    moe.tokens_combine(s["out_rows"], s["pos"], s["mix"], s["y"], **kw)
    moe.block_norm(s["x"], s["y"], s["res"], normed=s["nxt"], stats=s["st"], rows_per_gate=s["per"], **{n: s[n] for n in PARAMS}, **kw)


def backward(s, stream=None):
    kw = dict(stream=stream)
    x = dict(codes=s["xc"], scales=s["xs"]) if "codes" in s else dict(x=s["rows"])
    moe.block_norm_backward(s["d_res"], s["x"], s["y"], s["st"], s["d_x"], s["d_y"], d_normed=s["d_next"], rows_per_gate=s["per"],
                            **{n: s[n] for n in PARAMS}, **{"d_" + n: s["d_" + n] for n in PARAMS}, **kw)
    moe.tokens_combine_backward(s["d_y"], s["out_rows"], s["pos"], s["mix"], s["d_rows"], s["d_mix"], **kw)
    moe.experts_hidden_backward(s["d_rows"], s["offsets"], s["wd"], s["d_pre"], hidden=s["hid2"], pre=s.get("pre"),
                                codes=s.get("codes"), scales=s.get("scales"), **kw)
    moe.experts_product_backward(s["d_rows"], s["offsets"], s["wd"], x=s["hid2"], d_w=s["d_wd"], **kw)
    moe.experts_product_backward(s["d_pre"], s["offsets"], s["w"], d_x=s["d_xr"], d_w=s["d_w"], **x, **kw)
    moe.tokens_dispatch_backward(s["d_xr"], s["pos"], s["d_n0"], **kw)
    # the gradient of x: through the first norm, on top of the residual's
    moe.block_norm_backward(s["d_x"], s["x"], None, s["st0"], s["d_total"], None, d_normed=s["d_n0"], w_pre=s["w_pre0"],
                            d_w_pre=s["d_w_pre0"], **kw)


GRADS = ("d_total", "d_w", "d_wd", "d_mix", "d_w_pre0", "d_w_post", "d_gate", "d_alpha", "d_w_pre")


def step64(s):
    """The same step in float64: (res, nxt) and the gradients by torch's autograd."""
    leaf = {n: s[n].double().cpu().requires_grad_() for n in ("x", "w", "wd", "mix", "w_pre0", "w_post", "gate", "alpha", "w_pre")}
    x = leaf["x"]
    rms = lambda v: torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)  # noqa: E731
    n0 = leaf["w_pre0"] * x / rms(x)
    y = []
    ids = s["ids"].cpu().numpy()
    for i in range(x.shape[0]):
        row = torch.zeros(H, dtype=torch.float64)
        for j in range(k):
            e = ids[i, j]
            if e >= 0:
                p = leaf["w"][e] @ n0[i]
                h = torch.nn.functional.silu(p[:I]) * p[I:]
                row = row + leaf["mix"][i, j] * (leaf["wd"][e] @ h)
        y.append(row)
    y = torch.stack(y)
    res = leaf["alpha"] * x + leaf["gate"][torch.arange(x.shape[0]) // s["per"]] * (leaf["w_post"] * y / rms(y))
    nxt = leaf["w_pre"] * res / rms(res)
    total = (res * s["d_res"].double().cpu()).sum() + (nxt * s["d_next"].double().cpu()).sum()
    g = dict(zip(leaf, torch.autograd.grad(total, list(leaf.values()))))
    return res.detach(), nxt.detach(), {**{"d_" + n: v for n, v in g.items()}, "d_total": g["x"]}


@pytest.mark.parametrize("dtype,keep", [("f32", "type"), ("f32", "8 bits"), ("f16", "type"), ("bf16", "8 bits"), ("bf16", "type")])
def test_training_step(dtype, keep):
    """2-norms.  A result has passed about 8 roundings to its type; the rows with few terms of the fp32 sums add 2^-20.  Kept in
    8 bits, x, g and u are each off by up to 1/127 of their block's largest: 2^-7 sqrt(3) of the values' root mean
    square and less (a uniform error is a third of its bound; a block's largest is about 2.5 times its root mean square)."""
    s = tensors(dtype, keep)
    forward(s)
    backward(s)
    res, nxt, g = step64(s)
    tol = 8 * torch.finfo(DTYPES[dtype]).eps / 2 + 2.0 ** -20
    for n, ref in (("res", res), ("nxt", nxt)):
        assert np.linalg.norm(f64(s[n]) - ref.numpy()) <= tol * np.linalg.norm(ref.numpy()), n
    if keep == "8 bits":
        tol += 2.0 ** -7 * 3 ** 0.5
    for n in GRADS:
        ref = g[n].numpy()
        assert np.linalg.norm(f64(s[n]) - ref) <= tol * np.linalg.norm(ref), (n, np.linalg.norm(f64(s[n]) - ref) / np.linalg.norm(ref))


def test_gradients_against_differences():
    """The fp32 step's gradients along random directions against differences of its own forward pass."""
    s = tensors("f32", "type", seed=40)
    forward(s)
    backward(s)

    def value():
        forward(s)
        return float((s["res"].double() * s["d_res"].double()).sum() + (s["nxt"].double() * s["d_next"].double()).sum())

    for n, grad in (("x", "d_total"), ("w", "d_w"), ("wd", "d_wd"), ("mix", "d_mix"), ("w_pre0", "d_w_pre0"), ("w_post", "d_w_post"),
                    ("gate", "d_gate"), ("alpha", "d_alpha"), ("w_pre", "d_w_pre")):
        v, g = s[n].clone(), s[grad].double().clone()
        d = g.float() / g.norm().float()   # the steepest direction: the difference is the gradient's own norm
        h = 2e-3 * float(v.norm()) / v.numel() ** 0.5
        ends = []
        for sign in (1, -1):
            s[n].copy_(v + sign * h * d)
            ends.append(value())
        s[n].copy_(v)
        num = (ends[0] - ends[1]) / (2 * h)
        # values are sums of 2 T H products of numbers of size 1 with fp32 errors of about 2^-21 each, at random: 3e-5; h^2's term is
        # under 1e-4 of the gradient at such steps
        assert abs(num - float((g * d.double()).sum())) <= 2e-3 * float(g.norm()) + 1e-4 / h, n


@pytest.mark.parametrize("keep", ["type", "8 bits"])
def test_captured_step(keep):
    """Captured once, replayed with new inputs, eager work and synchronizations between: every replay as the eager step."""
    s, e = tensors("bf16", keep, seed=60, T=700), tensors("bf16", keep, seed=60, T=700)
    forward(s)
    backward(s)   # the library's code is loaded before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(s)
        backward(s)
    for r in range(4):
        for n in ("x", "d_res", "d_next"):
            v = randn(100 + 3 * r, *s[n].shape, dtype=s[n].dtype)
            s[n].copy_(v)
            e[n].copy_(v)
        new = torch.from_numpy(picks(200 + r, 700, k, E, 0.2 * (r % 3))).cuda()
        s["ids"].copy_(new)
        e["ids"].copy_(new)
        graph.replay()
        forward(e)
        backward(e)
        torch.cuda.synchronize()
        live = int(e["offsets"][-1])
        for n in ("res", "nxt", "offsets", *GRADS):
            assert torch.equal(s[n], e[n]), (r, n)
        assert torch.equal(s["hid"][:live], e["hid"][:live])


def test_two_graphs_share_a_workspace():
    """Two captured calls that use one workspace, replayed one after the other, either way round."""
    R, K, M = 6000, 128, 192
    off = torch.tensor([0, R], dtype=torch.int32).cuda()
    need = moe.gpu_lib().moe_experts_product_workspace(R, K, M, 1)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    w = torch.empty(1, M, K, dtype=torch.bfloat16, device="cuda")
    sets = [(randn(i, R, M, dtype=torch.bfloat16), randn(i + 5, R, K, dtype=torch.bfloat16), torch.empty(1, M, K, device="cuda")) for i in (1, 2)]
    want = []
    for d, x, d_w in sets:
        moe.experts_product_backward(d, off, w, x=x, d_w=d_w)
        want.append(d_w.clone())
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    torch.cuda.synchronize()
    for graph, (d, x, d_w) in zip(graphs, sets):
        with torch.cuda.graph(graph):
            moe.experts_product_backward(d, off, w, x=x, d_w=d_w, workspace=ws)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for _, _, d_w in sets:
            d_w.fill_(7)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(sets[i][2], want[i])


def test_streams_and_two_calls_at_once():
    a, b = tensors("f16", "8 bits", seed=1, T=900), tensors("f16", "8 bits", seed=2, T=900)
    want = []
    for s in (a, b):
        forward(s)
        backward(s)
        want.append({n: s[n].clone() for n in ("res", "nxt", *GRADS)})
        for n in ("res", "nxt", *GRADS):
            s[n].fill_(9)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for s, stream in ((a, one), (b, two.cuda_stream)):
        forward(s, stream)
        backward(s, stream)
    torch.cuda.synchronize()
    for s, v in zip((a, b), want):
        for n in v:
            assert torch.equal(s[n], v[n]), n


def test_single_tokens_give_the_rows_of_a_prompt():
    """A decode step of one token: within a rounding of the same token in a longer call (another tile, another order of sums)."""
    t, R = torch.bfloat16, 400
    x, w, wd = randn(1, R, H, dtype=t), randn(2, 1, 2 * I, H, dtype=t, std=H ** -0.5), randn(3, 1, H, I, dtype=t, std=I ** -0.5)
    h, out = torch.empty(R, I, dtype=t, device="cuda"), torch.empty(R, H, dtype=t, device="cuda")
    moe.experts_hidden(x, torch.tensor([0, R], dtype=torch.int32).cuda(), w, h)
    one, off = torch.empty(1, I, dtype=t, device="cuda"), torch.tensor([0, 1], dtype=torch.int32).cuda()
    for i in (0, 7, R - 1):
        moe.experts_hidden(x[i:i + 1], off, w, one)
        # equal, or the neighbouring number where the sums' last bits meet a border
        assert ((one - h[i]).abs() <= torch.finfo(t).eps * h[i].abs()).all()


def test_outputs_count_as_modified_and_inputs_do_not():
    s = tensors("f32", "8 bits")
    s2 = tensors("f32", "type")
    for v in (s, s2):
        before = {n: t._version for n, t in v.items() if isinstance(t, torch.Tensor)}
        forward(v)
        backward(v)
        inputs = ("x", "w", "wd", "mix", "w_pre0", "w_post", "alpha", "w_pre", "gate", "ids", "d_next", "d_res")
        for n in before:
            assert (v[n]._version > before[n]) == (n not in inputs), n


def test_refusals_of_the_binding():
    s = tensors("f32", "8 bits")
    bad = [
        lambda: moe.experts_hidden(s["rows"], s["offsets"], s["w"].half(), s["hid"]),
        lambda: moe.experts_hidden(s["rows"], s["offsets"], s["w"][:, :2 * I - 2], s["hid"]),
        lambda: moe.experts_hidden(s["rows"], s["offsets"].long(), s["w"], s["hid"]),
        lambda: moe.experts_hidden(s["rows"], s["offsets"], s["w"], s["hid"], codes=s["codes"]),
        lambda: moe.experts_hidden(s["rows"], s["offsets"], s["w"], s["hid"], codes=s["codes"], scales=s["scales"][:, 1:]),
        lambda: moe.experts_hidden(s["rows"], s["offsets"], s["w"], s["hid"], activation="relu"),
        lambda: moe.experts_hidden(s["rows"].cpu(), s["offsets"], s["w"], s["hid"]),
        lambda: moe.experts_hidden(s["rows"].t(), s["offsets"], s["w"], s["hid"]),
        lambda: moe.experts_product(s["hid"], s["offsets"], s["wd"], s["hid"]),
        lambda: moe.experts_product(s["hid"].double(), s["offsets"], s["wd"], s["out_rows"]),
        lambda: moe.experts_hidden_backward(s["d_rows"], s["offsets"], s["wd"], s["d_pre"]),
        lambda: moe.experts_product_backward(s["d_rows"], s["offsets"], s["wd"], d_w=s["d_wd"]),
        lambda: moe.experts_product_backward(s["d_rows"], s["offsets"], s["wd"], x=s["hid"], d_w=s["d_wd"].half()),
        lambda: moe.rows_encode(s["rows"], s["xc"], s["xs"][:, :-1]),
        lambda: moe.rows_encode(s["rows"], s["xc"].float(), s["xs"]),
        lambda: moe.block_norm(s["x"], s["y"], s["res"], w_pre=s["w_pre"]),
        lambda: moe.block_norm(s["x"], s["y"], s["res"], gate=s["gate"], rows_per_gate=0),
        lambda: moe.block_norm(s["x"], s["y"], s["res"], gate=s["gate"], rows_per_gate=T),
        lambda: moe.block_norm(s["x"], s["y"], s["res"], w_post=s["w_post"].half()),
        lambda: moe.block_norm(s["x"], s["y"], s["res"], eps=-1.0),
        lambda: moe.block_norm_backward(s["d_res"], s["x"], s["y"], None, s["d_x"], s["d_y"], w_post=s["w_post"]),
        lambda: moe.block_norm_backward(s["d_res"], s["x"], s["y"], s["st"], s["d_x"], s["d_y"], d_gate=s["d_gate"]),
    ]
    before = {n: t.clone() for n, t in s.items() if isinstance(t, torch.Tensor)}
    for i, call in enumerate(bad):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code in (moe.ERR_INVALID, moe.ERR_UNSUPPORTED), i
    torch.cuda.synchronize()
    for n, t in before.items():
        assert torch.equal(s[n], t), n


def test_oracle_step_agrees():
    """The float64 oracle's functions chained give the step that autograd differentiates."""
    s = tensors("f32", "type", seed=9)
    forward(s)
    ids = s["ids"].cpu().numpy()
    order = ot.order(ids, E)
    n0 = o.norm(f64(s["x"]), w_pre=f64(s["w_pre0"]))[1]
    rows = ot.dispatch(n0, order, np.zeros((T * k, H)))
    h, _ = o.hidden(rows, order["offsets"], f64(s["w"]), "silu", np.zeros((T * k, I)), np.zeros((T * k, 2 * I)))
    y = ot.combine(o.product(h, order["offsets"], f64(s["wd"]), np.zeros((T * k, H))), order["pos"], f64(s["mix"]))
    res = o.norm(f64(s["x"]), y, per=s["per"], **{n: f64(s[n]) for n in PARAMS})[0]
    assert np.allclose(res, step64(s)[0].numpy(), rtol=1e-12, atol=1e-12)
    assert np.linalg.norm(f64(s["res"]) - res) <= 8 * 2.0 ** -24 * 8 * np.linalg.norm(res)
