"""Large dispatches that copy rows: the counts of slices together with the copy, several rounds of tokens a
workgroup, and slices beyond the 64th."""
import numpy as np
import pytest
import torch

import expert_offload_lru_amd as moe
from token_harness import DTYPES, order_buffers, place, randn

pytestmark = pytest.mark.gpu


def order(ids, E):
    """Sorted by (expert, pick) with a stable sort: what oracle/tokens.py does pick by pick."""
    T, k = ids.shape
    flat = ids.reshape(-1).astype(np.int64)
    valid = (flat >= 0) & (flat < E)
    key = np.where(valid, flat, E)
    src = np.argsort(key, kind="stable")
    R = int(valid.sum())
    pos = np.full(T * k, -1)
    pos[src[:R]] = np.arange(R)
    src[R:] = -1
    return dict(offsets=np.searchsorted(np.sort(flat[valid]), np.arange(E + 1)), pos=pos.reshape(T, k), src=src,
                expert=np.where(src >= 0, flat[src], -1)), R


def some_ids(T, k, E, drop):
    rng = np.random.default_rng(T + k)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    return ids


# T, k, E, H, dtype, dropped: a whole workgroup a token and five to eight tokens; groups of 64, 16 and 8 lanes; odd rows
@pytest.mark.parametrize("T,k,E,H,dt,drop", [
    (1025, 8, 128, 2048, "bf16", 0.0), (6000, 4, 60, 1024, "bf16", 0.05), (8192, 8, 128, 520, "f32", 0.0),
    (6001, 8, 300, 1001, "f16", 0.1), (20000, 3, 64, 100, "f32", 0.0), (20011, 2, 16, 72, "bf16", 0.3),
    (33000, 1, 5, 33, "f16", 0.0), (5000, 16, 1024, 300, "bf16", 0.02)])
def test_rows_of_many_tokens(T, k, E, H, dt, drop):
    dtype, ids = DTYPES[dt], some_ids(T, k, E, drop)
    x = randn(T, T, H, dtype=dtype)
    rows, o = torch.full((T * k, H), 3.0, dtype=dtype, device="cuda"), order_buffers(T, k, E)
    moe.tokens_dispatch(x, torch.from_numpy(ids).cuda(), E, rows, **o)
    want, R = order(ids, E)
    for name, v in want.items():
        assert np.array_equal(o[name].cpu().numpy(), v), name
    src = torch.from_numpy(want["src"][:R]).cuda()
    assert torch.equal(rows[:R], x[src // k])           # copied bit by bit
    assert (rows[R:] == 3.0).all()


def test_strided_rows_of_many_tokens():
    T, k, E, H, ld, offset = 5000, 3, 20, 75, 83, 1
    ids = some_ids(T, k, E, 0.1)
    x = randn(5, T, H, dtype=torch.bfloat16, ld=ld, offset=offset)
    rows = place(torch.full((T * k, H), 3.0, dtype=torch.bfloat16, device="cuda"), ld, offset)
    o = order_buffers(T, k, E)
    moe.tokens_dispatch(x, torch.from_numpy(ids).cuda(), E, rows, **o)
    want, R = order(ids, E)
    src = torch.from_numpy(want["src"][:R]).cuda()
    assert torch.equal(rows[:R], x[src // k]) and (rows[R:] == 3.0).all()
    outside = rows._base.clone()
    outside[offset:offset + T * k * ld].view(T * k, ld)[:, :H] = 7.0
    assert (outside == 7.0).all()          # nothing written beside the rows


@pytest.mark.parametrize("T,k,E", [(300001, 8, 128), (2200003, 1, 40)])
def test_order_of_millions_of_picks(T, k, E):
    ids, o = some_ids(T, k, E, 0.05), order_buffers(T, k, E)
    moe.tokens_dispatch(None, torch.from_numpy(ids).cuda(), E, None, **o)
    for name, v in order(ids, E)[0].items():
        assert np.array_equal(o[name].cpu().numpy(), v), name
