"""Experts' feed-forward, rows kept in 8 bits and block norms in float64, from their definitions."""
import numpy as np

BLOCK = 32


def encode(x):
    """(codes, scales) of the rows of x: column c is codes * 2^(scales - 133); 255: the block held inf or NaN."""
    R, C = x.shape
    nb = -(-C // BLOCK)
    codes, scales = np.zeros((R, C), np.int64), np.zeros((R, nb), np.int64)
    for b in range(nb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK].astype(np.float64)
        for i in range(R):
            top = np.max(np.abs(v[i]))
            if not np.isfinite(top):
                scales[i, b] = 255
                continue
            e = -133
            if top > 0:
                e = max(-133, int(np.floor(np.log2(top))) - 8)
                while np.rint(top * 2.0 ** -e) > 127 and e < 121:
                    e += 1
            codes[i, b * BLOCK:(b + 1) * BLOCK] = np.clip(np.rint(v[i] * 2.0 ** -e), -127, 127)
            scales[i, b] = e + 133
    return codes, scales


def decode(codes, scales, largest=np.inf):
    at = np.arange(codes.shape[1]) // BLOCK
    s = scales.astype(np.float64)[:, at]
    return np.where(s == 255, np.nan, np.clip(codes * 2.0 ** (s - 133), -largest, largest))


def segments(offsets, n_rows):
    """(expert, first row, end) of every expert: an offset counts as at least those before it."""
    out, run = [], min(max(int(offsets[0]), 0), n_rows)
    for e in range(len(offsets) - 1):
        end = max(run, min(max(int(offsets[e + 1]), 0), n_rows))
        out.append((e, run, end))
        run = end
    return out


def act(g, kind):
    """The activation and its slope."""
    if kind == "silu":
        p = 1 / (1 + np.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    c = np.sqrt(2 / np.pi)
    t = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def product(x, offsets, w, out):
    """out with the experts' rows replaced by W_e x."""
    out = out.astype(np.float64).copy()
    for e, a, b in segments(offsets, x.shape[0]):
        out[a:b] = x[a:b].astype(np.float64) @ w[e].astype(np.float64).T
    return out


def product_backward(d_out, x, offsets, w, d_x):
    """(d_x with the experts' rows replaced, d_w)."""
    d_x, d_w = d_x.astype(np.float64).copy(), np.zeros(w.shape)
    for e, a, b in segments(offsets, d_out.shape[0]):
        d_x[a:b] = d_out[a:b].astype(np.float64) @ w[e].astype(np.float64)
        d_w[e] = d_out[a:b].astype(np.float64).T @ x[a:b].astype(np.float64)
    return d_x, d_w


def hidden(x, offsets, w, kind, rows, pre):
    """(rows, pre) with the experts' rows replaced by act(g) u and [g, u]."""
    I = w.shape[1] // 2
    pre = product(x, offsets, w, pre)
    rows = rows.astype(np.float64).copy()
    for _, a, b in segments(offsets, x.shape[0]):
        rows[a:b] = act(pre[a:b, :I], kind)[0] * pre[a:b, I:]
    return rows, pre


def hidden_backward(d_out, offsets, w, pre, kind, d_pre, rows):
    """(d_pre, hidden, d_h) with the experts' rows replaced."""
    I = w.shape[2]
    d_pre, rows = d_pre.astype(np.float64).copy(), rows.astype(np.float64).copy()
    d_h = np.zeros((d_out.shape[0], I))
    for e, a, b in segments(offsets, d_out.shape[0]):
        d_h[a:b] = d_out[a:b].astype(np.float64) @ w[e].astype(np.float64)
        g, u = pre[a:b, :I].astype(np.float64), pre[a:b, I:].astype(np.float64)
        v, slope = act(g, kind)
        d_pre[a:b] = np.concatenate([d_h[a:b] * u * slope, d_h[a:b] * v], 1)
        rows[a:b] = v * u
    return d_pre, rows, d_h


def _gate_rows(gate, per, R):
    return 1.0 if gate is None else gate.astype(np.float64)[np.arange(R) // per]


def norm(x, y=None, w_post=None, gate=None, per=1, alpha=None, w_pre=None, eps=1e-6):
    """(out, normed, r_y, r_out); what is not asked for is None or 0."""
    x = x.astype(np.float64)
    R = x.shape[0]
    r_y, r_o, normed = np.zeros(R), np.zeros(R), None
    out = x
    if y is not None:
        z = y.astype(np.float64)
        if w_post is not None:
            r_y = 1 / np.sqrt(np.mean(z * z, 1) + eps)
            z = w_post.astype(np.float64) * (z * r_y[:, None])
        out = x * (1.0 if alpha is None else alpha.astype(np.float64)) + _gate_rows(gate, per, R) * z
    if w_pre is not None:
        r_o = 1 / np.sqrt(np.mean(out * out, 1) + eps)
        normed = w_pre.astype(np.float64) * (out * r_o[:, None])
    return out, normed, r_y, r_o


def norm_backward(d_out, d_normed, x, y, r_y, r_o, w_post=None, gate=None, per=1, alpha=None, w_pre=None):
    """dict of d_x, d_y, d_w_post, d_gate, d_alpha, d_w_pre from the inverse roots of the forward pass."""
    x = x.astype(np.float64)
    R, H = x.shape
    y = np.zeros((R, H)) if y is None else y.astype(np.float64)
    a = 1.0 if alpha is None else alpha.astype(np.float64)
    g = _gate_rows(gate, per, R)
    wp = 1.0 if w_post is None else w_post.astype(np.float64)
    r_y = np.ones((R, 1)) if w_post is None else r_y.reshape(R, 1).astype(np.float64)
    r_o = r_o.reshape(R, 1).astype(np.float64)
    z = y * r_y
    out = x * a + g * wp * z
    D = np.zeros((R, H)) if d_out is None else d_out.astype(np.float64)
    got = {}
    if d_normed is not None:
        dn = d_normed.astype(np.float64)
        t = w_pre.astype(np.float64) * dn
        D = D + r_o * t - out * r_o ** 3 * np.mean(t * out, 1, keepdims=True)
        got["d_w_pre"] = np.sum(dn * out * r_o, 0)
    c = g * wp * D
    got["d_x"] = a * D
    got["d_y"] = c if w_post is None else r_y * c - y * r_y ** 3 * np.mean(c * y, 1, keepdims=True)
    got["d_alpha"] = np.sum(D * x, 0)
    got["d_w_post"] = np.sum(g * D * z, 0)
    dg = wp * D * z
    got["d_gate"] = np.stack([dg[i:i + per].sum(0) for i in range(0, R, per)]) if R else np.zeros((0, H))
    return got
