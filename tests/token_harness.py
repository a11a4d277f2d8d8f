"""Inputs and tolerances of the token-order and adapter tests.  (Test infrastructure.)

A tolerance counts roundings.  A value rounded to type t is off by at most eps(t)/2 of itself (half
of t's smallest step near zero); an fp32 sum of n terms, in whatever order, by at most n 2^-24 of the
sum of the terms' sizes, and 2^-23 instead where a matrix instruction adds, which may cut instead
of round.
"""
import numpy as np
import torch

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().cpu().double().numpy()


def assert_near(got, ref, dtype, slack):
    """|got - ref| <= eps/2 |ref| + slack (elementwise; slack: the fp32 error before the rounding)."""
    info = torch.finfo(dtype)
    got = f64(got)
    slack = np.asarray(slack)
    tol = info.eps / 2 * (np.abs(ref) + slack) + slack + info.smallest_normal * info.eps / 2
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float(err[bad].max()) if np.isfinite(err[bad]).all() else "not finite",
                           [tuple(map(int, i)) for i in np.argwhere(bad)[:4]])


def assert_norm(got, ref, dtype, terms, more=0.0):
    """2-norm of the error: the rounding at the end, and 4 sqrt(terms) 2^-24 for sums whose roundings
    are independent (a term that is lost or counted twice is off by 1/sqrt(terms))."""
    n = np.linalg.norm(ref)
    if n == 0:
        assert not np.any(f64(got))
        return
    tol = torch.finfo(dtype).eps / 2 + 4 * np.sqrt(terms) * 2.0 ** -24 + more
    assert np.linalg.norm(f64(got) - ref) <= tol * n, np.linalg.norm(f64(got) - ref) / n


def randn(seed, *shape, dtype=torch.float32, std=1.0, ld=None, offset=0):
    """A seeded normal matrix on the GPU; ld and offset place it inside a wider, oddly aligned buffer."""
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(shape, generator=g) * std).to(dtype).cuda()
    if ld is None and not offset:
        return v
    return place(v, ld or shape[-1], offset)


def place(v, ld, offset=0):
    buf = torch.full((offset + v.shape[0] * ld + 16,), 7.0, dtype=v.dtype, device="cuda")
    view = buf[offset:offset + v.shape[0] * ld].view(v.shape[0], ld)[:, :v.shape[1]]
    view.copy_(v)
    return view


def picks(seed, T, k, E, drop=0.0):
    """Distinct experts a token, some of them dropped (-1)."""
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32) if T else np.zeros((0, k), np.int32)
    if drop:
        ids = np.where(rng.random((T, k)) < drop, -1, ids).astype(np.int32)
    return ids


def order_buffers(T, k, E):
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(offsets=torch.full((E + 1,), -7, **i32), pos=torch.full((T, k), -7, **i32),
                src=torch.full((T * k,), -7, **i32), expert=torch.full((T * k,), -7, **i32))
