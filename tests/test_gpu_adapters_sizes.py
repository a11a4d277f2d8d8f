"""Adapters at sizes that reach the variants of the block kernels which test_gpu_adapters.py leaves out, with
tolerances of fp32 sums and the results' roundings alone."""
import numpy as np
import pytest
import torch

import expert_offload_lru_amd as moe
from oracle import tokens as ref
from test_gpu_adapters import backward, check_backward, forward, forward_slack, make, numbers, sizes
from token_harness import assert_near, assert_norm

pytestmark = pytest.mark.gpu

# T, n, r, inner, outer, dtype, wtype, order of the rows' adapters
SHAPES = [
    # fp32 adapters and activations in blocks: 16 rows with ranks to 16, 32, 64 and over; 32 rows
    (1100, 3, 16, 128, 96, "f32", "f32", "runs"),
    (1300, 40, 20, 72, 100, "f32", "f32", "mixed"),
    (1100, 3, 60, 64, 72, "f32", "f32", "runs"),
    (2100, 4, 90, 64, 64, "f32", "f32", "mixed"),
    (4200, 5, 32, 64, 72, "f32", "f32", "runs"),
    (4300, 3, 40, 72, 64, "f32", "f32", "mixed"),
    # ranks 17 to 32 beside fp32 activations, few and many rows
    (300, 3, 24, 128, 96, "f32", "f32", "mixed"),
    (400, 5, 32, 72, 64, "f32", "bf16", "runs"),
    (1500, 6, 24, 64, 136, "f32", "f16", "mixed"),
    (4200, 3, 30, 64, 64, "f32", "bf16", "runs"),
    # the gradients' blocks of 32 rows: just below, at and above their threshold
    (16383, 4, 32, 64, 64, "bf16", "bf16", "runs"),
    (16384, 4, 32, 64, 64, "bf16", "bf16", "runs"),
    (16385, 70, 32, 64, 72, "bf16", "bf16", "mixed"),
    (8200, 3, 64, 64, 72, "bf16", "bf16", "runs"),
    (8192, 3, 64, 64, 64, "f32", "f32", "runs"),
    (16390, 5, 32, 64, 64, "f32", "bf16", "mixed"),
    (5300, 2, 100, 64, 64, "bf16", "bf16", "runs"),
    (16400, 3, 40, 64, 40, "f16", "f16", "mixed"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_forward(shape):
    s = make(*shape, seed=1100)
    m, dtype = numbers(s), s["x"].dtype
    got = forward(s, base=s["base"])
    want = ref.adapters(m["x"], m["adapter"], m["a"], m["b"], m["scale"], m["base"])
    assert_near(got, want, dtype, forward_slack(m, torch.float32, True))
    assert_norm(got, want, dtype, shape[3] + shape[2])
    none = s["adapter"] < 0
    assert torch.equal(got[none], s["base"][none])


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_backward(shape):
    """d_a and d_b are fp32, and nothing on their way or d_x's is rounded to less."""
    T, n, r, inner, outer = shape[:5]
    s = make(*shape, seed=1200)
    m, dtype = numbers(s), s["x"].dtype
    z = sizes(m)
    got = backward(s, dx_base=s["dx_base"])
    want = ref.adapters_backward(m["d_out"], m["x"], m["adapter"], m["a"], m["b"], m["scale"], m["dx_base"])
    size = ref.adapters_backward(z["d_out"], z["x"], m["adapter"], z["a"], z["b"], z["scale"])
    slack = [(outer + r + 16) * 2.0 ** -23 * size[0] + 2.0 ** -24 * z["dx_base"],
             (outer + T + 16) * 2.0 ** -23 * size[1], (inner + T + 16) * 2.0 ** -23 * size[2]]
    for g, w, e, of, terms in zip(got, want, slack, (dtype, torch.float32, torch.float32), (outer + r, outer + T, inner + T)):
        assert_near(g, w, of, e)
        assert_norm(g, w, of, terms)


@pytest.mark.parametrize("dt,wt", [("f32", "f32"), ("f32", "f16"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("T", [30, 1300])
def test_matrices_inside_one_buffer(T, dt, wt):
    """a and b at any element of a packed buffer of parameters."""
    n, r, inner, outer = 3, 16, 64, 72
    s = make(T, n, r, inner, outer, dt, wt, "mixed", seed=1300)
    m, dtype = numbers(s), s["x"].dtype
    packed = torch.full((s["a"].numel() + s["b"].numel() + 4,), float("nan"), dtype=s["a"].dtype, device="cuda")
    at = 1 + s["a"].numel()
    t = dict(s, a=packed[1:at].view_as(s["a"]), b=packed[at + 2:at + 2 + s["b"].numel()].view_as(s["b"]))
    t["a"].copy_(s["a"])
    t["b"].copy_(s["b"])
    want = ref.adapters(m["x"], m["adapter"], m["a"], m["b"], m["scale"], m["base"])
    assert_near(forward(t, base=s["base"]), want, dtype, forward_slack(m, dtype, True))
    check_backward(s, m, backward(t, dx_base=s["dx_base"]), True)


def test_rows_in_the_order_of_a_dispatch():
    """An adapter an expert on dispatched rows: 128 of them over 4096 picks, the rows behind the last without one."""
    T, k, n, r, inner, outer = 512, 8, 128, 16, 64, 72
    rng = np.random.default_rng(7)
    ids = np.argsort(rng.random((T, n)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    flat = np.sort(ids.reshape(-1))
    expert = np.concatenate([flat[flat >= 0], flat[flat < 0]]).astype(np.int32)
    s = make(T * k, n, r, inner, outer, "bf16", "bf16", "runs", seed=1400)
    s["adapter"] = torch.from_numpy(expert).cuda()
    m = numbers(s)
    want = ref.adapters(m["x"], m["adapter"], m["a"], m["b"], m["scale"])
    assert_near(forward(s), want, torch.bfloat16, forward_slack(m, torch.bfloat16, False))
    check_backward(s, m, backward(s), False)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,n,r", [(1, 6, 64), (300, 20, 24), (512, 40, 16)])
def test_workspace_of_few_rows_is_enough(T, n, r, dt):
    """Nothing is written behind the bytes that a call of few rows asks for."""
    s = make(T, n, r, 64, 72, dt, dt, "mixed", seed=1500)
    need = moe.gpu_lib().moe_adapters_workspace(T, 64, 72, n, r)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    check_backward(s, numbers(s), backward(s, workspace=ws[:need]), False)
    assert (ws[need:] == 0xFF).all()
