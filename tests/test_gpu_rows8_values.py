"""Every code with every scale of rows kept in 8 bits, against their definition (oracle/experts.py): exact."""
import numpy as np
import pytest
import torch

import expert_offload_lru_amd as moe
from oracle import experts as o
from token_harness import DTYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_code_and_scale(dtype):
    """A value beyond the type's largest finite one is read as that; scale 255 is NaN."""
    t = DTYPES[dtype]
    codes = np.tile(np.arange(-128, 128), (256, 1))
    scales = np.repeat(np.arange(256)[:, None], 8, 1)
    x = torch.full((256, 256), 7.0, dtype=t, device="cuda")
    moe.rows_decode(torch.from_numpy(codes).to(torch.int8).cuda(), torch.from_numpy(scales).to(torch.uint8).cuda(), x)
    want = torch.from_numpy(o.decode(codes, scales, torch.finfo(t).max)).to(t)
    assert torch.equal(torch.nan_to_num(x.cpu(), nan=1.5), torch.nan_to_num(want, nan=1.5)) and torch.isfinite(x[:255]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [64, 61])
def test_least_code_in_a_weight_gradient(M, dtype):
    """-128 times the largest scale: d_w from codes has the bits of d_w from the values read back, and is finite."""
    t, R, N = DTYPES[dtype], 40, 72
    codes = torch.full((R, M), -128, dtype=torch.int8, device="cuda")
    scales = torch.full((R, 2), 254, dtype=torch.uint8, device="cuda")
    d = torch.zeros(R, N, dtype=t, device="cuda")
    d[3], d[17] = 0.25, -0.5
    back, w = torch.empty(R, M, dtype=t, device="cuda"), torch.empty(1, N, M, dtype=t, device="cuda")
    moe.rows_decode(codes, scales, back)
    off = torch.tensor([0, R], dtype=torch.int32).cuda()
    a, b = torch.empty(1, N, M, device="cuda"), torch.empty(1, N, M, device="cuda")
    moe.experts_product_backward(d, off, w, codes=codes, scales=scales, d_w=a)
    moe.experts_product_backward(d, off, w, x=back, d_w=b)
    assert torch.equal(a, b) and torch.isfinite(a).all() and (a == torch.finfo(t).max / 4).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_how_far_values_are_off(dtype):
    """By 1/127 of the block's largest size; by 2^-134 where that is under 2^-127."""
    t = DTYPES[dtype]
    g = torch.Generator().manual_seed(3)
    x = torch.randn(300, 96, generator=g, dtype=torch.float64)
    tops = torch.randint(-149, 128, (300, 3), generator=g).double()
    tops[:40], tops[40:80] = torch.arange(-149, -109)[:, None].double(), torch.arange(88, 128)[:, None].double()
    x = (x.view(300, 3, 32) / x.view(300, 3, 32).abs().amax(-1, keepdim=True) * 1.99 * 2.0 ** tops[..., None]).reshape(300, 96).to(t)
    x[250:, ::32] = torch.finfo(t).max
    assert torch.isfinite(x).all()
    codes, scales = torch.empty(300, 96, dtype=torch.int8, device="cuda"), torch.empty(300, 3, dtype=torch.uint8, device="cuda")
    back = torch.empty(300, 96, dtype=t, device="cuda")
    moe.rows_encode(x.cuda(), codes, scales)
    moe.rows_decode(codes, scales, back)
    v = x.double().view(300, 3, 32)
    off, top = (back.cpu().double().view(300, 3, 32) - v).abs().amax(-1), v.abs().amax(-1)
    assert (off <= torch.where(top >= 2.0 ** -127, top / 127, torch.full_like(top, 2.0 ** -134))).all()
    largest = codes.cpu().view(300, 3, 32).abs().amax(-1)
    assert ((largest >= 64) | (top < 2.0 ** -127)).all()
