"""Argument checks of include/moe_experts.h that return before any HIP call (CPU): addresses are only compared."""
import pytest

import expert_offload_lru_amd as moe
from test_capi_symbols import _declared, _exported

M = 1 << 20   # addresses M apart do not overlap at these sizes
INV, UNS = moe.ERR_INVALID, moe.ERR_UNSUPPORTED


def test_every_declared_function_is_exported():
    declared = set(_declared("moe_experts.h"))
    assert not declared - _exported(moe.LIB_PATH)
    assert {"moe_experts_hidden", "moe_block_norm_backward", "moe_rows_decode"} <= declared


def call(name, base, change):
    rc = getattr(moe.gpu_lib(), name)(*{**base, **change}.values())
    assert rc == moe.OK or moe.gpu_lib().moe_last_error()
    return rc


ENCODE = dict(x=M, ld_x=40, dtype=0, n_rows=4, cols=40, codes=2 * M, ld_codes=40, scales=3 * M, ld_scales=2, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(dtype=3), INV), (dict(n_rows=-1), INV), (dict(cols=0), INV), (dict(cols=1 << 24, ld_x=1 << 24, ld_codes=1 << 24), UNS),
    (dict(n_rows=1 << 24), UNS), (dict(x=None), INV), (dict(codes=None), INV), (dict(scales=None), INV), (dict(ld_x=39), INV),
    (dict(ld_codes=39), INV), (dict(ld_scales=1), INV), (dict(codes=M + 639), INV), (dict(scales=2 * M + 159), INV),
    (dict(ld_x=1 << 41), INV), (dict(n_rows=0), moe.OK),
])
def test_encode_and_decode(change, rc):
    assert call("moe_rows_encode", ENCODE, change) == rc
    decode = {n: {**ENCODE, **change}[n] for n in ("codes", "ld_codes", "scales", "ld_scales", "dtype", "n_rows", "cols", "x",
                                                    "ld_x", "stream")}
    if "scales" not in change or change["scales"] is None:   # inputs of decode may overlap
        assert moe.gpu_lib().moe_rows_decode(*decode.values()) == rc


HIDDEN = dict(x=M, ld_x=8, dtype=2, n_rows=4, inner=8, inter=40, offsets=2 * M, n_experts=3, w=3 * M, activation=0, hidden=4 * M,
              ld_hidden=40, pre=None, ld_pre=0, codes=6 * M, ld_codes=80, scales=7 * M, ld_scales=4, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(dtype=-1), INV), (dict(n_rows=-1), INV), (dict(inner=0), INV), (dict(inter=0), INV), (dict(n_experts=0), INV),
    (dict(n_experts=1025), UNS), (dict(n_rows=1 << 24), UNS), (dict(inner=1 << 24), UNS), (dict(inter=1 << 23), UNS),
    (dict(n_rows=(1 << 24) - 1, inter=1 << 22), UNS), (dict(activation=2), INV), (dict(activation=-1), INV), (dict(x=None), INV),
    (dict(offsets=None), INV), (dict(w=None), INV), (dict(hidden=None), INV), (dict(pre=5 * M, ld_pre=80), INV),
    (dict(codes=None), INV), (dict(scales=None), INV), (dict(ld_x=7), INV), (dict(ld_hidden=39), INV), (dict(ld_codes=79), INV),
    (dict(ld_scales=3), INV), (dict(pre=5 * M, ld_pre=79, codes=None, scales=None), INV), (dict(hidden=M), INV),
    (dict(hidden=3 * M + 2 * 3 * 80 * 8 - 2), INV), (dict(codes=4 * M + 100), INV), (dict(scales=2 * M), INV), (dict(n_rows=0), moe.OK),
])
def test_hidden(change, rc):
    assert call("moe_experts_hidden", HIDDEN, change) == rc


BACK = dict(d_out=M, ld_d_out=8, dtype=2, n_rows=4, outer=8, inter=40, offsets=2 * M, n_experts=3, w=3 * M, activation=1, pre=None,
            ld_pre=0, codes=6 * M, ld_codes=80, scales=7 * M, ld_scales=4, d_pre=8 * M, ld_d_pre=80, hidden=9 * M, ld_hidden=40,
            stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(d_out=None), INV), (dict(w=None), INV), (dict(offsets=None), INV), (dict(d_pre=None), INV), (dict(codes=None, scales=None), INV),
    (dict(pre=5 * M, ld_pre=80), INV), (dict(scales=None), INV), (dict(ld_d_pre=79), INV), (dict(ld_hidden=39), INV), (dict(ld_d_out=7), INV),
    (dict(d_pre=6 * M), INV), (dict(d_pre=M), INV), (dict(hidden=8 * M + 600), INV), (dict(hidden=7 * M), INV), (dict(activation=7), INV),
    (dict(dtype=3), INV), (dict(n_experts=1025), UNS), (dict(n_rows=0), moe.OK),
    (dict(pre=5 * M, ld_pre=80, codes=None, scales=None, d_pre=5 * M), INV),
])
def test_hidden_backward(change, rc):
    assert call("moe_experts_hidden_backward", BACK, change) == rc


PRODUCT = dict(x=M, ld_x=8, dtype=0, n_rows=4, inner=8, outer=16, offsets=2 * M, n_experts=3, w=3 * M, out=4 * M, ld_out=16, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(x=None), INV), (dict(offsets=None), INV), (dict(w=None), INV), (dict(out=None), INV), (dict(ld_x=7), INV), (dict(ld_out=15), INV),
    (dict(out=M), INV), (dict(out=3 * M + 4), INV), (dict(out=2 * M + 12), INV), (dict(dtype=4), INV), (dict(outer=0), INV),
    (dict(outer=1 << 24, ld_out=1 << 24), UNS), (dict(n_rows=-2), INV), (dict(n_rows=0), moe.OK),
])
def test_product(change, rc):
    assert call("moe_experts_product", PRODUCT, change) == rc


PRODUCT_BACK = dict(d_out=M, ld_d_out=16, dtype=0, n_rows=4, inner=8, outer=16, offsets=2 * M, n_experts=3, w=3 * M, x=4 * M, ld_x=8,
                    codes=None, ld_codes=0, scales=None, ld_scales=0, d_x=5 * M, ld_d_x=8, d_w=6 * M, workspace=None,
                    workspace_bytes=0, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(d_out=None), INV), (dict(offsets=None), INV), (dict(w=None), INV), (dict(x=None), INV), (dict(ld_d_out=15), INV), (dict(ld_x=7), INV),
    (dict(ld_d_x=7), INV), (dict(codes=7 * M, ld_codes=8, scales=8 * M, ld_scales=1), INV), (dict(x=None, codes=7 * M, ld_codes=8), INV),
    (dict(x=None, codes=7 * M, ld_codes=7, scales=8 * M, ld_scales=1), INV), (dict(d_x=M), INV), (dict(d_w=5 * M), INV), (dict(d_w=3 * M), INV),
    (dict(d_x=4 * M), INV), (dict(d_x=None, d_w=None), moe.OK), (dict(n_experts=1025), UNS),
    (dict(n_rows=9000, n_experts=1), INV),                                                                  # a workspace is wanted
    (dict(n_rows=9000, n_experts=1, workspace=30 * M + 8, workspace_bytes=M), INV),
    (dict(n_rows=9000, n_experts=1, workspace=6 * M, workspace_bytes=M), INV),
])
def test_product_backward(change, rc):
    assert call("moe_experts_product_backward", PRODUCT_BACK, change) == rc


NORM = dict(x=M, ld_x=8, y=2 * M, ld_y=8, dtype=0, n_rows=4, hidden=8, w_post=3 * M, gate=4 * M, rows_per_gate=2, alpha=5 * M, w_pre=6 * M,
            eps=1e-6, out=7 * M, ld_out=8, normed=8 * M, ld_normed=8, stats=9 * M, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(dtype=3), INV), (dict(n_rows=-1), INV), (dict(hidden=0), INV), (dict(hidden=16385), UNS), (dict(n_rows=1 << 24), UNS),
    (dict(n_rows=1 << 23, hidden=8193), UNS), (dict(rows_per_gate=0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(x=None), INV), (dict(y=None), INV), (dict(w_pre=None), INV), (dict(normed=None), INV),
    (dict(ld_x=7), INV), (dict(ld_y=7), INV), (dict(ld_out=7), INV), (dict(ld_normed=7), INV), (dict(out=M + 4), INV), (dict(out=M, ld_out=9), INV),
    (dict(normed=7 * M), INV), (dict(stats=6 * M + 28), INV), (dict(stats=M), INV), (dict(out=4 * M), INV), (dict(normed=3 * M), INV),
    (dict(out=None, normed=None, w_pre=None, stats=None), INV), (dict(n_rows=0), moe.OK),
])
def test_norm(change, rc):
    assert call("moe_block_norm", NORM, change) == rc


NORM_BACK = dict(d_out=M, ld_d_out=8, d_normed=2 * M, ld_d_normed=8, x=3 * M, ld_x=8, y=4 * M, ld_y=8, dtype=0, n_rows=4, hidden=8, w_post=5 * M,
                 gate=6 * M, rows_per_gate=2, alpha=7 * M, w_pre=8 * M, stats=9 * M, d_x=10 * M, ld_d_x=8, d_y=11 * M, ld_d_y=8, d_w_post=12 * M,
                 d_gate=13 * M, d_alpha=14 * M, d_w_pre=15 * M, workspace=16 * M, workspace_bytes=M, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(x=None), INV), (dict(y=None), INV), (dict(stats=None), INV), (dict(d_out=None, d_normed=None), INV), (dict(w_post=None), INV),
    (dict(gate=None), INV), (dict(alpha=None), INV), (dict(w_pre=None, d_w_pre=None), INV), (dict(workspace=None), INV),
    (dict(workspace_bytes=64), INV), (dict(workspace=16 * M + 4), INV), (dict(workspace=M), INV), (dict(d_x=M + 8), INV), (dict(d_x=M, ld_d_x=9), INV),
    (dict(d_y=10 * M), INV), (dict(d_gate=12 * M), INV), (dict(d_w_post=5 * M), INV), (dict(d_alpha=3 * M), INV), (dict(rows_per_gate=0), INV),
    (dict(ld_d_x=7), INV), (dict(hidden=20000), UNS),
])
def test_norm_backward(change, rc):
    assert call("moe_block_norm_backward", NORM_BACK, change) == rc


def test_workspaces():
    lib = moe.gpu_lib()
    assert lib.moe_experts_product_workspace(100, 64, 64, 4) == 0
    assert lib.moe_experts_product_workspace(9000, 64, 64, 1) > 0
    assert lib.moe_experts_product_workspace(9000, 64, 64, 2000) == 0
    assert lib.moe_experts_product_workspace(-1, 64, 64, 1) == 0
    assert lib.moe_block_norm_workspace(100, 64, 0) > 0 and lib.moe_block_norm_workspace(100, 64, 7) > 0
    assert lib.moe_block_norm_workspace(100, 20000, 1) == 0


@pytest.mark.parametrize("n_rows,width,rc", [((1 << 24) - 1, 1 << 12, INV), ((1 << 24) - 1, 1 << 13, UNS), (1 << 20, 1 << 16, INV),
                                             (1 << 20, 1 << 17, UNS), ((1 << 24) - 1, 7, INV)])
def test_more_than_a_launch_holds(n_rows, width, rc):
    """Refused before the tensors are looked at (they are NULL here)."""
    none = dict(x=None, ld_x=width, dtype=2, n_rows=n_rows, inner=64, outer=width, offsets=None, n_experts=4, w=None, out=None,
                ld_out=width, stream=None)
    assert moe.gpu_lib().moe_experts_product(*none.values()) == rc
    assert moe.gpu_lib().moe_experts_product(*{**none, "inner": width, "outer": 64}.values()) == rc


@pytest.mark.parametrize("n_rows,E,inner,outer,rc", [
    # (n_rows / 128 + min(n_rows, E)) * ceil(w / 64) < 2^24 - 16
    (1024, 1024, 8, 64 * 16256, INV), (1024, 1024, 8, 64 * 16256 + 1, UNS), (1151, 1024, 8, 64 * 16256, INV), (1152, 1024, 8, 64 * 16256, UNS),
    (1024, 1024, 8, 1 << 22, UNS), (1, 1024, 8, 1 << 20, INV), ((1 << 24) - 1, 1, 64, 64 * 127, INV), ((1 << 24) - 1, 1, 64, 64 * 128, UNS),
    # widths under 8: (n_rows / 64 + min(n_rows, E)) * ceil(w / 32) < 2^25 - 32
    (65280, 4, 7, 32 * 32767, INV), (65280, 4, 7, 32 * 32767 + 1, UNS), (65343, 4, 7, 32 * 32767, INV), (65344, 4, 7, 32 * 32767, UNS),
    # E * ceil(inner / 128) * ceil(outer / 128) < 2^24 - 16
    (1, 1024, 127 * 128, 129 * 128, INV), (1, 1024, 127 * 128, 129 * 128 + 1, UNS), (1, 1024, 128 * 128, 128 * 128, UNS),
])
def test_what_the_workgroups_of_one_launch_can_be(n_rows, E, inner, outer, rc):
    """The documented limits, on either side; refused before the tensors are looked at (they are NULL here)."""
    lib = moe.gpu_lib()
    for a, b in ((inner, outer), (outer, inner)):
        none = dict(x=None, ld_x=a, dtype=1, n_rows=n_rows, inner=a, outer=b, offsets=None, n_experts=E, w=None)
        assert lib.moe_experts_product(*none.values(), None, b, None) == rc
        assert lib.moe_experts_hidden(*none.values(), 0, None, b, None, 0, None, 0, None, 0, None) == rc
        assert lib.moe_experts_hidden_backward(*none.values(), 0, None, 0, None, 0, None, 0, None, 0, None, 0, None) == rc
        assert lib.moe_experts_product_backward(*none.values(), None, 0, None, 0, None, 0, None, a, 64, None, 0, None) == rc


def test_activation_names():
    from expert_offload_lru_amd import experts
    assert experts._activation("silu") == 0 and experts._activation("gelu") == 1
    with pytest.raises(moe.MoeError) as e:
        experts._activation("relu")
    assert e.value.code == INV
