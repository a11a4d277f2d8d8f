"""Block norms through the C entry points, as a program without the torch binding calls them, against float64
(oracle/experts.py).  Tolerances as in test_gpu_block_norm.py.
"""
import numpy as np
import pytest
import torch

import expert_offload_lru_amd as moe
from oracle import experts as o
from test_gpu_block_norm import R5, forward, oracle_of, params, sizes
from token_harness import assert_near, f64, randn

pytestmark = pytest.mark.gpu


def backward_c(d_out, d_n, x, y, p, stats, rows_per_gate):
    """moe_block_norm_backward with every gradient; p as block_norm takes it."""
    lib, (R, H) = moe.gpu_lib(), x.shape
    d_x, d_y = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    g = {n: torch.full_like(p[n], 7.0) for n in ("w_post", "gate", "alpha", "w_pre")}
    need = lib.moe_block_norm_workspace(R, H, rows_per_gate)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    a = lambda t: t.data_ptr()  # noqa: E731
    rc = lib.moe_block_norm_backward(a(d_out), H, a(d_n), H, a(x), H, a(y), H, moe.T_F32, R, H, a(p["w_post"]), a(p["gate"]),
                                     rows_per_gate, a(p["alpha"]), a(p["w_pre"]), a(stats), a(d_x), H, a(d_y), H, a(g["w_post"]),
                                     a(g["gate"]), a(g["alpha"]), a(g["w_pre"]), a(ws), need, torch.cuda.current_stream().cuda_stream)
    assert rc == moe.OK, lib.moe_last_error()
    return d_x, d_y, g


@pytest.mark.parametrize("rows_per_gate", [0, 1, 2048, 2 ** 31 - 1])   # 0: as many as there are rows, 1: one more
@pytest.mark.parametrize("R,H", [(1, 64), (2, 64), (3, 512), (1, 513), (1, 1024), (3, 1024), (5, 500), (1, 4096), (40, 200)])
def test_one_gate_for_fewer_rows_than_it_may_have(R, H, rows_per_gate):
    per = rows_per_gate if rows_per_gate > 1 else R + rows_per_gate
    x, y, d_out, d_n = (randn(i, R, H) for i in (1, 2, 21, 22))
    p = params(H, R, 1, 1, 1, 1, R)
    stats = forward(x, y, p)[2]
    d_x, d_y, g = backward_c(d_out, d_n, x, y, p, stats, per)
    q, s = oracle_of(p), f64(stats)
    v = [f64(t) for t in (d_out, d_n, x, y)]
    ref = o.norm_backward(*v, s[:, 0], s[:, 1], **q)
    big = sizes(*(np.abs(t) for t in v), s[:, 0], s[:, 1], **{n: t if n == "per" else np.abs(t) for n, t in q.items()})
    assert_near(d_x, ref["d_x"], torch.float32, R5 * big["d_x"])
    assert_near(d_y, ref["d_y"], torch.float32, R5 * big["d_y"])
    for n, t in g.items():
        assert_near(t, ref["d_" + n], torch.float32, (R5 + R * 2.0 ** -24) * big["d_" + n])
