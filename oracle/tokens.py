"""Token order, combine and low-rank adapters in float64, from their definitions."""
import numpy as np


def order(ids, n_experts):
    """Valid picks by (expert, pick): dict of offsets, pos, src, expert (-1 behind the last row)."""
    T, k = ids.shape
    picks = [(int(e), p) for p, e in enumerate(ids.reshape(-1)) if 0 <= e < n_experts]
    picks.sort()
    offsets = np.zeros(n_experts + 1, dtype=np.int64)
    pos, src, expert = (np.full(T * k, -1, dtype=np.int64) for _ in range(3))
    for row, (e, p) in enumerate(picks):
        offsets[e + 1:] += 1
        pos[p], src[row], expert[row] = row, p, e
    return dict(offsets=offsets, pos=pos.reshape(T, k), src=src, expert=expert)


def dispatch(x, o, rows):
    """rows with row pos[t, j] = x[t]; other rows as given."""
    rows = rows.copy()
    T, k = o["pos"].shape
    for t in range(T):
        for j in range(k):
            if o["pos"][t, j] >= 0:
                rows[o["pos"][t, j]] = x[t]
    return rows


def combine(rows, pos, gate=None, base=None):
    T, k = pos.shape
    out = np.zeros((T, rows.shape[1])) if base is None else base.astype(np.float64).copy()
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < rows.shape[0]:
                out[t] += (1.0 if gate is None else float(gate[t, j])) * rows[pos[t, j]].astype(np.float64)
    return out


def combine_backward(d_out, rows, pos, gate, d_rows):
    """(d_rows with the picks' rows replaced, d_gate)."""
    T, k = pos.shape
    d_rows, d_gate = d_rows.astype(np.float64).copy(), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = pos[t, j]
            if 0 <= p < rows.shape[0]:
                d_rows[p] = float(gate[t, j]) * d_out[t].astype(np.float64)
                d_gate[t, j] = np.dot(d_out[t].astype(np.float64), rows[p].astype(np.float64))
    return d_rows, d_gate


def adapters(x, adapter, a, b, scale, base=None):
    T, outer = x.shape[0], b.shape[1]
    out = np.zeros((T, outer)) if base is None else base.astype(np.float64).copy()
    for i in range(T):
        e = adapter[i]
        if 0 <= e < a.shape[0]:
            v = a[e].astype(np.float64) @ x[i].astype(np.float64)
            out[i] += float(scale[e]) * (b[e].astype(np.float64) @ v)
    return out


def adapters_backward(d_out, x, adapter, a, b, scale, dx_base=None):
    """(d_x, d_a, d_b)."""
    T, inner = x.shape
    d_x = np.zeros((T, inner)) if dx_base is None else dx_base.astype(np.float64).copy()
    d_a, d_b = np.zeros(a.shape), np.zeros(b.shape)
    for i in range(T):
        e = adapter[i]
        if 0 <= e < a.shape[0]:
            ae, be = a[e].astype(np.float64), b[e].astype(np.float64)
            xi, dy = x[i].astype(np.float64), d_out[i].astype(np.float64)
            u = float(scale[e]) * (be.T @ dy)
            d_x[i] += ae.T @ u
            d_a[e] += np.outer(u, xi)
            d_b[e] += float(scale[e]) * np.outer(dy, ae @ xi)
    return d_x, d_a, d_b
