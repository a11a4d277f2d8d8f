"""The token and adapter operators beside torch's autograd: outputs count as modified in place."""
import pytest
import torch

import expert_offload_lru_amd as moe
from token_harness import order_buffers, randn

pytestmark = pytest.mark.gpu

T, k, E, H, r = 6, 2, 5, 16, 4


def tensors():
    s = dict(x=randn(1, T, H), gate=randn(2, T, k), a=randn(3, E, r, H), b=randn(4, E, H, r), scale=randn(5, E))
    s["ids"] = (torch.arange(T * k, device="cuda", dtype=torch.int32) % E).view(T, k)
    s.update(order_buffers(T, k, E), rows=torch.zeros(T * k, H, device="cuda"), prod=torch.zeros(T * k, H, device="cuda"),
             out=torch.zeros(T, H, device="cuda"), d_out=randn(6, T, H), d_prod=torch.zeros(T * k, H, device="cuda"),
             d_gate=torch.zeros(T, k, device="cuda"), d_rows=torch.zeros(T * k, H, device="cuda"),
             d_x=torch.zeros(T, H, device="cuda"), d_a=torch.zeros(E, r, H, device="cuda"), d_b=torch.zeros(E, H, r, device="cuda"))
    return s


STEPS = [
    (("rows", "offsets", "pos", "src", "expert"), lambda s: moe.tokens_dispatch(
        s["x"], s["ids"], E, s["rows"], s["offsets"], s["pos"], s["src"], s["expert"])),
    (("offsets", "pos", "src", "expert"), lambda s: moe.tokens_dispatch(
        None, s["ids"], E, None, s["offsets"], s["pos"], s["src"], s["expert"])),
    (("prod",), lambda s: moe.adapters_forward(s["rows"], s["expert"], s["a"], s["b"], s["scale"], s["prod"])),
    (("out",), lambda s: moe.tokens_combine(s["prod"], s["pos"], s["gate"], s["out"])),
    (("d_prod", "d_gate"), lambda s: moe.tokens_combine_backward(
        s["d_out"], s["prod"], s["pos"], s["gate"], s["d_prod"], s["d_gate"])),
    (("d_rows", "d_a", "d_b"), lambda s: moe.adapters_backward(
        s["d_prod"], s["rows"], s["expert"], s["a"], s["b"], s["scale"], s["d_rows"], s["d_a"], s["d_b"])),
    (("d_x",), lambda s: moe.tokens_dispatch_backward(s["d_rows"], s["pos"], s["d_x"])),
]


def test_every_output_counts_as_modified_and_no_input_does():
    s = tensors()
    for outputs, call in STEPS:
        before = {n: t._version for n, t in s.items()}
        call(s)
        for n, t in s.items():
            assert (t._version > before[n]) == (n in outputs), n


def test_a_graph_that_kept_an_output_refuses_to_run_backward_on_new_values():
    s = tensors()
    STEPS[0][1](s)
    w = torch.ones(T, H, device="cuda", requires_grad=True)
    y = (w * s["out"]).sum()
    STEPS[3][1](s)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_in_inference_mode():
    with torch.inference_mode():
        s = tensors()
        for _, call in STEPS:
            call(s)
    t = tensors()
    for _, call in STEPS:
        call(t)
    for n in s:
        assert torch.equal(s[n], t[n]), n
