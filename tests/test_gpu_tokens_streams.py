"""Calls on a stream given as an object, with a workspace of the call's own that belongs to it."""
import pytest
import torch

import expert_offload_lru_amd as moe
from test_gpu_adapters import backward, forward, make

pytestmark = pytest.mark.gpu


def test_adapters_on_a_given_stream():
    s = make(1400, 6, 24, 250, 320, "bf16", "bf16", "runs", seed=1600)
    want, wantb = forward(s, base=s["base"]), backward(s)
    out, d_x = torch.empty_like(want), torch.empty_like(wantb[0])
    d_a, d_b = torch.empty_like(wantb[1]), torch.empty_like(wantb[2])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        for t in (out, d_x, d_a, d_b):
            t.fill_(9.0)
        side.wait_stream(torch.cuda.current_stream())
        moe.adapters_forward(s["x"], s["adapter"], s["a"], s["b"], s["scale"], out, base=s["base"], stream=stream)
        moe.adapters_backward(s["d_out"], s["x"], s["adapter"], s["a"], s["b"], s["scale"], d_x, d_a, d_b, stream=stream)
        side.synchronize()
        assert torch.equal(out, want)
        for g, w in zip((d_x, d_a, d_b), wantb):
            assert torch.equal(g, w)
