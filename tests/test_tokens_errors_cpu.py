"""Argument checks of include/moe_tokens.h that return before any HIP call (CPU): addresses are only compared."""
import pytest
import torch

import expert_offload_lru_amd as moe
from test_capi_symbols import _declared, _exported

M = 1 << 20   # addresses M apart do not overlap at these sizes
INV, UNS = moe.ERR_INVALID, moe.ERR_UNSUPPORTED


def test_every_declared_function_is_exported():
    assert not set(_declared("moe_tokens.h")) - _exported(moe.LIB_PATH)
    assert "moe_adapters_backward" in _declared("moe_tokens.h")


DISPATCH = dict(x=M, ld_x=8, dtype=0, n_tokens=4, hidden=8, ids=2 * M, top_k=2, n_experts=5, rows=3 * M, ld_rows=8,
                offsets=4 * M, pos=5 * M, src=6 * M, expert=7 * M, workspace=None, workspace_bytes=0, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(dtype=3), INV), (dict(dtype=-1), INV), (dict(n_tokens=-1), INV), (dict(top_k=0), INV), (dict(n_experts=0), INV),
    (dict(top_k=17), UNS), (dict(n_experts=1025), UNS), (dict(n_tokens=1 << 24), UNS), (dict(hidden=0), INV),
    (dict(hidden=1 << 24, ld_x=1 << 24, ld_rows=1 << 24), UNS),
    (dict(ld_x=7), INV), (dict(ld_rows=7), INV), (dict(ld_rows=1 << 41), INV), (dict(ids=None), INV), (dict(offsets=None), INV),
    (dict(pos=None), INV), (dict(src=None), INV), (dict(expert=None), INV), (dict(x=None), INV), (dict(rows=None), INV),
    (dict(rows=M + 4), INV), (dict(pos=3 * M + 100), INV), (dict(src=5 * M + 28), INV), (dict(offsets=2 * M - 20), INV),
    (dict(n_tokens=5000, top_k=8, x=None, rows=None), INV),                               # a workspace is wanted
    (dict(n_tokens=5000, top_k=8, x=None, rows=None, workspace=9 * M + 2, workspace_bytes=1 << 20), INV),
])
def test_dispatch(change, rc):
    assert moe.gpu_lib().moe_tokens_dispatch(*{**DISPATCH, **change}.values()) == rc
    assert moe.gpu_lib().moe_last_error()


COMBINE = dict(rows=M, ld_rows=8, n_rows=8, dtype=2, n_tokens=4, hidden=8, pos=2 * M, gate=3 * M, top_k=2, base=4 * M,
               ld_base=8, out=5 * M, ld_out=8, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(rows=None), INV), (dict(pos=None), INV), (dict(gate=None), INV), (dict(out=None), INV), (dict(ld_out=7), INV),
    (dict(ld_base=7), INV), (dict(ld_rows=0), INV), (dict(out=4 * M, ld_out=9), INV), (dict(out=4 * M + 16), INV),
    (dict(out=M + 127), INV), (dict(n_rows=-1), INV), (dict(top_k=17), UNS), (dict(dtype=9), INV), (dict(n_tokens=-3), INV),
    (dict(n_tokens=0), moe.OK),
])
def test_combine(change, rc):
    assert moe.gpu_lib().moe_tokens_combine(*{**COMBINE, **change}.values()) == rc


def test_combine_backward_and_dispatch_backward():
    lib = moe.gpu_lib()
    back = dict(d_out=M, ld=8, rows=2 * M, ld_rows=8, n_rows=8, dtype=1, n_tokens=4, hidden=8, pos=3 * M, gate=4 * M,
                top_k=2, d_rows=5 * M, ld_d_rows=8, d_gate=6 * M, stream=None)
    for change in (dict(d_out=None), dict(d_gate=None), dict(d_rows=2 * M), dict(d_gate=4 * M), dict(ld_d_rows=3)):
        assert lib.moe_tokens_combine_backward(*{**back, **change}.values()) == INV
    assert lib.moe_tokens_combine_backward(*{**back, "n_tokens": 0}.values()) == moe.OK
    d = dict(d_rows=M, ld=8, n_rows=8, dtype=1, n_tokens=4, hidden=8, pos=3 * M, top_k=2, d_x=5 * M, ld_x=8, stream=None)
    for change in (dict(d_rows=None), dict(d_x=None), dict(d_x=M), dict(ld_x=1), dict(pos=None), dict(top_k=0)):
        assert lib.moe_tokens_dispatch_backward(*{**d, **change}.values()) == INV


FORWARD = dict(x=M, ld_x=8, base=2 * M, ld_base=16, dtype=0, n_rows=4, inner=8, outer=16, adapter=3 * M, a=4 * M, b=5 * M,
               wtype=2, scale=6 * M, n_adapters=3, rank=4, out=7 * M, ld_out=16,
               workspace=None, workspace_bytes=0, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(dtype=5), INV), (dict(wtype=5), INV), (dict(dtype=1), INV), (dict(dtype=1, wtype=0), INV), (dict(rank=0), INV),
    (dict(rank=257), UNS), (dict(inner=0), INV), (dict(outer=0), INV), (dict(n_adapters=0), INV), (dict(n_rows=-1), INV),
    (dict(n_rows=1 << 24), UNS), (dict(x=None), INV), (dict(adapter=None), INV), (dict(a=None), INV), (dict(b=None), INV),
    (dict(scale=None), INV), (dict(out=None), INV), (dict(ld_x=7), INV), (dict(ld_out=15), INV), (dict(ld_base=15), INV),
    (dict(out=M), INV), (dict(out=4 * M), INV), (dict(out=2 * M, ld_out=17), INV), (dict(n_rows=0), moe.OK),
    (dict(n_rows=2000), INV), (dict(n_rows=2000, workspace=9 * M, workspace_bytes=100), INV),   # a workspace is wanted
    (dict(n_rows=2000, workspace=9 * M + 8, workspace_bytes=M), INV), (dict(n_rows=2000, workspace=M, workspace_bytes=M), INV),
])
def test_adapters_forward(change, rc):
    assert moe.gpu_lib().moe_adapters_forward(*{**FORWARD, **change}.values()) == rc


BACKWARD = dict(d_out=8 * M, ld_d_out=16, x=M, ld_x=8, dx_base=2 * M, ld_dx_base=8, dtype=0, n_rows=4, inner=8, outer=16,
                adapter=3 * M, a=4 * M, b=5 * M, wtype=2, scale=6 * M, n_adapters=3, rank=4, d_x=7 * M, ld_d_x=8, d_a=9 * M,
                d_b=10 * M, workspace=11 * M, workspace_bytes=M, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(n_adapters=1025), UNS), (dict(d_a=None), INV), (dict(d_b=None), INV), (dict(d_out=None), INV), (dict(d_x=None), INV),
    (dict(d_x=M), INV), (dict(d_a=10 * M), INV), (dict(workspace=None), INV), (dict(workspace_bytes=8), INV),
    (dict(workspace=11 * M + 8), INV), (dict(workspace=M), INV), (dict(d_x=2 * M, ld_d_x=9), INV), (dict(rank=300), UNS),
])
def test_adapters_backward(change, rc):
    assert moe.gpu_lib().moe_adapters_backward(*{**BACKWARD, **change}.values()) == rc


def test_workspaces():
    lib = moe.gpu_lib()
    assert lib.moe_tokens_workspace(1, 8, 128) == 0
    assert lib.moe_tokens_workspace(1 << 20, 16, 1024) > 0
    assert lib.moe_tokens_workspace(-1, 8, 128) == 0
    assert lib.moe_adapters_workspace(100, 8, 8, 4, 300) == 0
    assert lib.moe_adapters_workspace(0, 8, 8, 4, 4) > 0
    assert lib.moe_adapters_forward_workspace(32, 2048, 2048, 8, 16) == 0
    assert lib.moe_adapters_forward_workspace_strided(32, 2048, 2048, 8, 16) == 0
    assert lib.moe_adapters_workspace_strided(100, 8, 8, 4, 300) == 0
    # room for copies, 4 bytes an element: of x and base and out; of x, d_out and d_x
    for name, copied in (("moe_adapters_forward_workspace", 2), ("moe_adapters_workspace", 3)):
        least, most = getattr(lib, name)(8192, 2048, 2048, 8, 16), getattr(lib, name + "_strided")(8192, 2048, 2048, 8, 16)
        assert most - least == copied * 8192 * 2048 * 4
        assert getattr(lib, name)(8192, 2047, 2047, 8, 16) == getattr(lib, name + "_strided")(8192, 2047, 2047, 8, 16)
    assert lib.moe_adapters_forward_workspace(8192, 2048, 2048, 8, 16) >= 8192 * 16 * 4


def test_sizes_that_the_library_cannot_hold():
    """Checked before ctypes cuts them to 32 bits."""
    from expert_offload_lru_amd import tokens
    assert tuple(tokens._dims("t", torch.zeros(1, 1).expand(2 ** 31 - 1, 5), 2)) == (2 ** 31 - 1, 5)
    for shape in ((2 ** 31, 1), (1, 2 ** 32 + 4)):
        with pytest.raises(moe.MoeError) as e:
            tokens._dims("t", torch.zeros(1, 1).expand(shape), 2)
        assert e.value.code == UNS
