"""Experts' feed-forward, rows kept in 8 bits and block norms: the binding of ``include/moe_experts.h``.

As in ``tokens.py``: every function takes torch tensors on one GPU, checks their shapes and types, and
enqueues the library's kernels on ``stream`` (default: the current stream of that GPU).  Outputs are tensors
that the caller holds; a matrix needs unit stride along its rows, vectors, weights, offsets, stats and fp32
gradients are contiguous.  ``MoeError`` with ``ERR_INVALID`` or ``ERR_UNSUPPORTED`` says what was refused.
Nothing is recorded by torch's autograd; outputs count as modified in place.

A row of an expert is row ``offsets[e] .. offsets[e+1]`` (int32 [E+1], as ``tokens_dispatch`` writes them; a
dense block is one expert); rows outside are not read, and left as they were.
"""
import torch

from . import gpu_lib
from .tokens import _array, _call, _dims, _matrix, _needed, _refuse, _type, _workspace

_ACTIVATIONS = {"silu": 0, "gelu": 1}
_F32, _I8, _U8, _I32 = torch.float32, torch.int8, torch.uint8, torch.int32


def _blocks(cols):
    return -(-cols // 32)


def _maybe_matrix(name, t, rows, cols, dtype, gpu):
    return (None, cols) if t is None else _matrix(name, t, rows, cols, dtype, gpu)


def _vector(name, t, H, gpu):
    return None if t is None else _array(name, t, (H,), _F32, gpu)


def _codes(codes, scales, rows, cols, blocks, gpu):
    """Addresses and row distances of codes and scales (None, if there are none)."""
    if codes is None and scales is None:
        return None, cols, None, blocks
    if codes is None or scales is None:
        _refuse("codes and scales go together")
    return _matrix("codes", codes, rows, cols, _I8, gpu) + _matrix("scales", scales, rows, blocks, _U8, gpu)


def _activation(name):
    code = _ACTIVATIONS.get(name)
    if code is None:
        _refuse(f"activation is {name!r}: one of {sorted(_ACTIVATIONS)} is wanted")
    return code


def _experts(offsets, gpu):
    """Number of experts and the address of offsets."""
    n = _dims("offsets", offsets, 1)[0]
    return n - 1, _array("offsets", offsets, (n,), _I32, gpu)


def _outputs(*tensors):
    return [t for t in tensors if t is not None]


def rows_encode(x, codes, scales, stream=None):
    """Keep x [R, C] in 8 bits (moe_rows_encode): codes int8 [R, C] and scales uint8 [R, ceil(C / 32)], a column's
    value being codes * 2^(scales - 133), 32 columns to a scale."""
    dtype, gpu = _type("x", x)
    R, C = _dims("x", x, 2)
    px, ldx = _matrix("x", x, R, C, x.dtype, gpu)
    _call(gpu_lib().moe_rows_encode, (codes, scales), gpu, stream, px, ldx, dtype, R, C,
          *_codes(codes, scales, R, C, _blocks(C), gpu))


def rows_decode(codes, scales, x, stream=None):
    """The values of rows kept in 8 bits, in x's type (moe_rows_decode)."""
    dtype, gpu = _type("x", x)
    R, C = _dims("x", x, 2)
    px, ldx = _matrix("x", x, R, C, x.dtype, gpu)
    _call(gpu_lib().moe_rows_decode, (x,), gpu, stream, *_codes(codes, scales, R, C, _blocks(C), gpu), dtype, R, C, px,
          ldx)


def experts_hidden(x, offsets, w, hidden, activation="silu", pre=None, codes=None, scales=None, stream=None):
    """hidden = act(x Wg^T) * (x Wu^T) for each expert's rows (moe_experts_hidden).

    x [R, inner], w [E, 2*inter, inner] (gate rows, then up rows), hidden [R, inter].  What the backward pass
    needs is kept in pre [R, 2*inter] of x's type, or in codes int8 [R, 2*inter] and scales uint8
    [R, 2*ceil(inter/32)] (the halves are blocked by themselves), or not at all.  activation: "silu", "gelu" (tanh).
    """
    dtype, gpu = _type("x", x)
    R, K = _dims("x", x, 2)
    E, p_off = _experts(offsets, gpu)
    I = _dims("hidden", hidden, 2)[1]
    px, ldx = _matrix("x", x, R, K, x.dtype, gpu)
    pw = _array("w", w, (E, 2 * I, K), x.dtype, gpu)
    ph, ldh = _matrix("hidden", hidden, R, I, x.dtype, gpu)
    pp, ldp = _maybe_matrix("pre", pre, R, 2 * I, x.dtype, gpu)
    _call(gpu_lib().moe_experts_hidden, _outputs(hidden, pre, codes, scales), gpu, stream, px, ldx, dtype, R, K, I, p_off, E,
          pw, _activation(activation), ph, ldh, pp, ldp, *_codes(codes, scales, R, 2 * I, 2 * _blocks(I), gpu))


def experts_hidden_backward(d_out, offsets, w, d_pre, hidden=None, activation="silu", pre=None, codes=None, scales=None,
                            stream=None):
    """Back through the down projection w [E, outer, inter] and the activation (moe_experts_hidden_backward).

    From d_out [R, outer] and what experts_hidden kept: d_pre [R, 2*inter], the gradient of [g, u], which
    is the d_out of experts_product_backward with experts_hidden's w; and hidden [R, inter] again, for the
    gradient of w (None: not wanted).
    """
    dtype, gpu = _type("d_out", d_out)
    R, H = _dims("d_out", d_out, 2)
    E, p_off = _experts(offsets, gpu)
    I = _dims("w", w, 3)[2]
    pd, ldd = _matrix("d_out", d_out, R, H, d_out.dtype, gpu)
    pw = _array("w", w, (E, H, I), d_out.dtype, gpu)
    pp, ldp = _maybe_matrix("pre", pre, R, 2 * I, d_out.dtype, gpu)
    pg, ldg = _matrix("d_pre", d_pre, R, 2 * I, d_out.dtype, gpu)
    ph, ldh = _maybe_matrix("hidden", hidden, R, I, d_out.dtype, gpu)
    _call(gpu_lib().moe_experts_hidden_backward, _outputs(d_pre, hidden), gpu, stream, pd, ldd, dtype, R, H, I, p_off, E, pw,
          _activation(activation), pp, ldp, *_codes(codes, scales, R, 2 * I, 2 * _blocks(I), gpu), pg, ldg, ph, ldh)


def experts_product(x, offsets, w, out, stream=None):
    """out = x W_e^T for each expert's rows (moe_experts_product); x [R, inner], w [E, outer, inner], out [R, outer]."""
    dtype, gpu = _type("x", x)
    R, K = _dims("x", x, 2)
    E, p_off = _experts(offsets, gpu)
    M = _dims("out", out, 2)[1]
    px, ldx = _matrix("x", x, R, K, x.dtype, gpu)
    pw = _array("w", w, (E, M, K), x.dtype, gpu)
    po, ldo = _matrix("out", out, R, M, x.dtype, gpu)
    _call(gpu_lib().moe_experts_product, (out,), gpu, stream, px, ldx, dtype, R, K, M, p_off, E, pw, po, ldo)


def experts_product_backward(d_out, offsets, w, x=None, codes=None, scales=None, d_x=None, d_w=None, workspace=None,
                             stream=None):
    """Gradients of experts_product (moe_experts_product_backward): d_x [R, inner] = d_out W_e, and d_w fp32
    [E, outer, inner] = sum of d_out x^T over each expert's rows; either may be None.  For d_w, x is given, or
    as kept in 8 bits (codes, scales).  workspace: any contiguous tensor of enough bytes, 16-byte aligned."""
    lib = gpu_lib()
    dtype, gpu = _type("d_out", d_out)
    R, M = _dims("d_out", d_out, 2)
    E, p_off = _experts(offsets, gpu)
    K = _dims("w", w, 3)[2]
    pd, ldd = _matrix("d_out", d_out, R, M, d_out.dtype, gpu)
    pw = _array("w", w, (E, M, K), d_out.dtype, gpu)
    px, ldx = _maybe_matrix("x", x, R, K, d_out.dtype, gpu)
    kept = _codes(codes, scales, R, K, _blocks(K), gpu)
    pg, ldg = _maybe_matrix("d_x", d_x, R, K, d_out.dtype, gpu)
    p_dw = None if d_w is None else _array("d_w", d_w, (E, M, K), _F32, gpu)
    if d_x is None and d_w is None:
        return
    need = _needed("moe_experts_product_workspace", R, K, M, E) if d_w is not None else 0
    ws = _workspace(need, workspace, gpu, stream) if need else None
    _call(lib.moe_experts_product_backward, _outputs(d_x, d_w), gpu, stream, pd, ldd, dtype, R, K, M, p_off, E, pw, px, ldx,
          *kept, pg, ldg, p_dw, ws.data_ptr() if need else None, ws.numel() * ws.element_size() if need else 0)


def _gates(gate, rows_per_gate, R, H, gpu):
    if rows_per_gate < 1:
        _refuse("rows_per_gate must be positive")
    return _array("gate", gate, (-(-R // rows_per_gate), H), _F32, gpu), min(rows_per_gate, max(R, 1))


def block_norm(x, y, out, w_post=None, gate=None, rows_per_gate=1, alpha=None, w_pre=None, normed=None, stats=None,
               eps=1e-6, stream=None):
    """out = alpha x + gate (w_post y r_y) and normed = w_pre out r_out (moe_block_norm), r the inverse root of a
    row's mean square plus eps.

    x, y, out, normed [R, H] of one type; w_post, alpha, w_pre fp32 [H]; gate fp32 [ceil(R / rows_per_gate), H]; stats
    fp32 [R, 2] for the backward pass.  Parameters that are None are left out (with w_pre goes normed); y
    (and out) None: the norm of x alone.  out and normed may each be x or y.
    """
    dtype, gpu = _type("x", x)
    R, H = _dims("x", x, 2)
    t = x.dtype
    px, ldx = _matrix("x", x, R, H, t, gpu)
    py, ldy = (None, H) if y is None else _matrix("y", y, R, H, t, gpu)
    po, ldo = (None, H) if out is None else _matrix("out", out, R, H, t, gpu)
    pn, ldn = (None, H) if normed is None else _matrix("normed", normed, R, H, t, gpu)
    pg, per = (None, 1) if gate is None else _gates(gate, rows_per_gate, R, H, gpu)
    p_stats = None if stats is None else _array("stats", stats, (R, 2), _F32, gpu)
    _call(gpu_lib().moe_block_norm, _outputs(out, normed, stats), gpu, stream, px, ldx, py, ldy, dtype, R, H,
          _vector("w_post", w_post, H, gpu), pg, per, _vector("alpha", alpha, H, gpu), _vector("w_pre", w_pre, H, gpu), eps,
          po, ldo, pn, ldn, p_stats)


def block_norm_backward(d_out, x, y, stats, d_x, d_y, d_normed=None, w_post=None, gate=None, rows_per_gate=1, alpha=None,
                        w_pre=None, d_w_post=None, d_gate=None, d_alpha=None, d_w_pre=None, workspace=None, stream=None):
    """Gradients of block_norm (moe_block_norm_backward) from d_out and d_normed (either may be None), with x, y, stats and the
    parameters of the forward call: d_x, d_y of x's type and fp32 gradients of the parameters; those that
    are None are not made.  d_x and d_y may each be one of d_out, d_normed, x and y."""
    lib = gpu_lib()
    dtype, gpu = _type("x", x)
    R, H = _dims("x", x, 2)
    t = x.dtype
    pd, ldd = (None, H) if d_out is None else _matrix("d_out", d_out, R, H, t, gpu)
    pn, ldn = (None, H) if d_normed is None else _matrix("d_normed", d_normed, R, H, t, gpu)
    px, ldx = _matrix("x", x, R, H, t, gpu)
    py, ldy = (None, H) if y is None else _matrix("y", y, R, H, t, gpu)
    pdx, lddx = (None, H) if d_x is None else _matrix("d_x", d_x, R, H, t, gpu)
    pdy, lddy = (None, H) if d_y is None else _matrix("d_y", d_y, R, H, t, gpu)
    pg, per = (None, 1) if gate is None else _gates(gate, rows_per_gate, R, H, gpu)
    p_stats = None if stats is None else _array("stats", stats, (R, 2), _F32, gpu)
    outputs = _outputs(d_x, d_y, d_w_post, d_gate, d_alpha, d_w_pre)
    if not outputs:
        return
    p_dgate = None
    if d_gate is not None:
        p_dgate = _array("d_gate", d_gate, (0, H) if gate is None else gate.shape, _F32, gpu)
    pw, wbytes = None, 0
    if d_w_post is not None or d_gate is not None or d_alpha is not None or d_w_pre is not None:
        ws = _workspace(_needed("moe_block_norm_workspace", R, H, per), workspace, gpu, stream)
        pw, wbytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _call(lib.moe_block_norm_backward, outputs, gpu, stream, pd, ldd, pn, ldn, px, ldx, py, ldy, dtype, R, H,
          _vector("w_post", w_post, H, gpu), pg, per, _vector("alpha", alpha, H, gpu), _vector("w_pre", w_pre, H, gpu), p_stats,
          pdx, lddx, pdy, lddy, _vector("d_w_post", d_w_post, H, gpu), p_dgate, _vector("d_alpha", d_alpha, H, gpu),
          _vector("d_w_pre", d_w_pre, H, gpu), pw, wbytes)
