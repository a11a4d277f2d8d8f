"""Token order and adapters: the binding of ``include/moe_tokens.h``.

Every function takes torch tensors on one GPU, checks their shapes and types, and enqueues the
library's kernels on ``stream`` (default: the current stream of that GPU).  Outputs are tensors that
the caller holds.  A matrix needs unit stride along its rows (a column slice of a wider matrix will
do); index, gate, scale, adapter and adapter-gradient tensors are contiguous.  ``MoeError`` with
``ERR_INVALID`` or ``ERR_UNSUPPORTED`` says what was refused; nothing is enqueued then.

Nothing here is recorded by torch's autograd: an output has no gradient, whether or not an input requires
one, and the ``_backward`` functions are the gradients, called by the training step (or from the ``backward``
of a ``torch.autograd.Function``).  Outputs count as modified in place.
"""
import functools

import torch

from . import ERR_INVALID, ERR_UNSUPPORTED, OK, T_BF16, T_F16, T_F32, MoeError, gpu_lib

_INT_MAX = 2 ** 31 - 1   # of the C sizes: ctypes would cut a larger number
_TYPES = {torch.float32: T_F32, torch.float16: T_F16, torch.bfloat16: T_BF16}

# torch.cuda.current_device() and .current_stream().cuda_stream without their Python layers (about 2 us a call)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                   or (lambda gpu: torch.cuda.current_stream(gpu).cuda_stream))
# tells torch's autograd of outputs written through their addresses, so that a graph that has kept one refuses to run
# backward on the new values (a third of torch.autograd.graph.increment_version's time)
_written = getattr(torch._C, "_increment_version", None) or torch.autograd.graph.increment_version


def _refuse(msg):
    raise MoeError(ERR_INVALID, msg)


# A call of few rows takes the GPU a few microseconds, so the checks are one comparison of what should
# be with what is for each tensor, and the words for what is wrong are found only then.

def _matrix(name, t, rows, cols, dtype, gpu):
    """Address and row distance of a [rows x cols] matrix."""
    if t.shape == (rows, cols) and t.dtype is dtype and t.get_device() == gpu:
        ld, unit = t.stride()
        if unit == 1 and ld >= cols:
            return t.data_ptr(), ld
        if cols > 1 and unit != 1:
            _refuse(f"{name} is not stored by rows")
        if ld < cols and rows > 1:
            _refuse(f"{name} has rows that overlap")
        return t.data_ptr(), max(ld, cols)
    _refuse(f"{name} must be a {dtype} tensor of shape {(rows, cols)} on GPU {gpu}, got {t.dtype} {tuple(t.shape)} "
            f"on {t.device}")


def _array(name, t, shape, dtype, gpu):
    if t.shape == shape and t.dtype is dtype and t.get_device() == gpu and t.is_contiguous():
        return t.data_ptr()
    _refuse(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on GPU {gpu}, "
            f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _dims(name, t, n):
    shape = t.shape
    if len(shape) != n:
        _refuse(f"{name} has {len(shape)} dimensions, not {n}")
    if max(shape) > _INT_MAX:
        raise MoeError(ERR_UNSUPPORTED, f"{name} has a size over {_INT_MAX}")
    return shape


def _type(name, t):
    """Type code and GPU of a tensor of values."""
    gpu = t.get_device()
    if gpu < 0:
        _refuse(f"{name} is on {t.device}, not a GPU")
    code = _TYPES.get(t.dtype)
    if code is None:
        _refuse(f"{name} is {t.dtype}: float32, float16 or bfloat16 is wanted")
    return code, gpu


def _call(fn, outputs, gpu, stream, *args):
    """The library call with `gpu` current and the stream's handle as last argument, writing the tensors of `outputs`."""
    if stream is not None and not isinstance(stream, int) and stream.device_index != gpu:
        _refuse(f"stream is one of GPU {stream.device_index}, the tensors are on GPU {gpu}")
    if _current_device() != gpu:
        with torch.cuda.device(gpu):
            return _call(fn, outputs, gpu, stream, *args)
    if stream is None:
        handle = _current_stream(gpu)
    else:
        handle = stream if isinstance(stream, int) else stream.cuda_stream
    rc = fn(*args, handle)
    if rc != OK:
        raise MoeError(rc, gpu_lib().moe_last_error().decode())
    _written(outputs)


@functools.lru_cache(maxsize=1024)
def _needed(fn, *sizes):
    """Workspace bytes of a call of these sizes."""
    return getattr(gpu_lib(), fn)(*sizes)


def _workspace(nbytes, given, gpu, stream):
    """A workspace tensor: the caller's, or a new one that belongs to the call's stream."""
    if given is not None:
        if given.get_device() != gpu or not given.is_contiguous():
            _refuse(f"workspace must be a contiguous tensor on GPU {gpu}")
        return given
    device = torch.device("cuda", gpu)
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    s = torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream
    with torch.cuda.stream(s):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def tokens_dispatch(x, ids, n_experts, rows, offsets, pos, src, expert, workspace=None, stream=None):
    """Tokens sorted by expert (moe_tokens_dispatch).

    x [T, H] and ids int32 [T, k] (-1: no pick) give rows [T*k, H] (as x), offsets int32
    [n_experts+1], pos int32 [T, k], src and expert int32 [T*k]: the valid picks p = t*k + j in the
    order of (ids[p], p) are rows 0 .. R-1; rows from R on are left as they were.  x = rows = None
    makes the order alone.
    """
    lib = gpu_lib()
    gpu = ids.get_device()
    if gpu < 0:
        _refuse(f"ids is on {ids.device}, not a GPU")
    T, k = _dims("ids", ids, 2)
    n = T * k
    if n_experts > _INT_MAX:
        raise MoeError(ERR_UNSUPPORTED, f"n_experts is over {_INT_MAX}")
    if (x is None) != (rows is None):
        _refuse("x and rows go together")
    i32 = torch.int32
    if x is None:
        dtype, H, px, ldx, pr, ldr = T_F32, 1, None, 1, None, 1
    else:
        dtype, H = _type("x", x)[0], _dims("x", x, 2)[1]
        px, ldx = _matrix("x", x, T, H, x.dtype, gpu)
        pr, ldr = _matrix("rows", rows, n, H, x.dtype, gpu)
    p_ids, p_off = _array("ids", ids, (T, k), i32, gpu), _array("offsets", offsets, (n_experts + 1,), i32, gpu)
    p_pos, p_src = _array("pos", pos, (T, k), i32, gpu), _array("src", src, (n,), i32, gpu)
    p_exp = _array("expert", expert, (n,), i32, gpu)
    need = _needed("moe_tokens_workspace", T, k, n_experts)
    ws = _workspace(need, workspace, gpu, stream) if need else None
    outputs = (offsets, pos, src, expert) if x is None else (rows, offsets, pos, src, expert)
    _call(lib.moe_tokens_dispatch, outputs, gpu, stream, px, ldx, dtype, T, H, p_ids, k, n_experts, pr, ldr, p_off, p_pos,
          p_src, p_exp, ws.data_ptr() if need else None, ws.numel() * ws.element_size() if need else 0)


def tokens_dispatch_backward(d_rows, pos, d_x, stream=None):
    """d_x[t] = sum_j d_rows[pos[t, j]] (moe_tokens_dispatch_backward)."""
    dtype, gpu = _type("d_rows", d_rows)
    (T, k), (R, H) = _dims("pos", pos, 2), _dims("d_rows", d_rows, 2)
    pr, ldr = _matrix("d_rows", d_rows, R, H, d_rows.dtype, gpu)
    px, ldx = _matrix("d_x", d_x, T, H, d_rows.dtype, gpu)
    p_pos = _array("pos", pos, (T, k), torch.int32, gpu)
    _call(gpu_lib().moe_tokens_dispatch_backward, (d_x,), gpu, stream, pr, ldr, R, dtype, T, H, p_pos, k, px, ldx)


def tokens_combine(rows, pos, gate, out, base=None, stream=None):
    """out[t] = base[t] + sum_j gate[t, j] rows[pos[t, j]] (moe_tokens_combine); base may be out."""
    dtype, gpu = _type("rows", rows)
    (T, k), (R, H) = _dims("pos", pos, 2), _dims("rows", rows, 2)
    pr, ldr = _matrix("rows", rows, R, H, rows.dtype, gpu)
    po, ldo = _matrix("out", out, T, H, rows.dtype, gpu)
    pb, ldb = (None, H) if base is None else _matrix("base", base, T, H, rows.dtype, gpu)
    p_pos = _array("pos", pos, (T, k), torch.int32, gpu)
    p_gate = _array("gate", gate, (T, k), torch.float32, gpu)
    _call(gpu_lib().moe_tokens_combine, (out,), gpu, stream, pr, ldr, R, dtype, T, H, p_pos, p_gate, k, pb, ldb, po, ldo)


def tokens_combine_backward(d_out, rows, pos, gate, d_rows, d_gate, stream=None):
    """d_rows[pos[t, j]] = gate[t, j] d_out[t] and d_gate[t, j] = <d_out[t], rows[pos[t, j]]>
    (moe_tokens_combine_backward); rows of d_rows that no pick names are left as they were."""
    dtype, gpu = _type("rows", rows)
    (T, k), (R, H) = _dims("pos", pos, 2), _dims("rows", rows, 2)
    pd, ldd = _matrix("d_out", d_out, T, H, rows.dtype, gpu)
    pr, ldr = _matrix("rows", rows, R, H, rows.dtype, gpu)
    pg, ldg = _matrix("d_rows", d_rows, R, H, rows.dtype, gpu)
    p_pos = _array("pos", pos, (T, k), torch.int32, gpu)
    p_gate = _array("gate", gate, (T, k), torch.float32, gpu)
    p_dgate = _array("d_gate", d_gate, (T, k), torch.float32, gpu)
    _call(gpu_lib().moe_tokens_combine_backward, (d_rows, d_gate), gpu, stream, pd, ldd, pr, ldr, R, dtype, T, H, p_pos,
          p_gate, k, pg, ldg, p_dgate)


def _adapter_shapes(a, b, gpu):
    n, r, inner = _dims("a", a, 3)
    outer = _dims("b", b, 3)[1]
    return (n, r, inner, outer, _array("a", a, (n, r, inner), a.dtype, gpu), _array("b", b, (n, outer, r), a.dtype, gpu),
            _type("a", a)[0])


def adapters_forward(x, adapter, a, b, scale, out, base=None, workspace=None, stream=None):
    """out[i] = base[i] + scale[e] B_e (A_e x[i]) with e = adapter[i] (moe_adapters_forward).

    x [T, inner], adapter int32 [T] (-1: none), a [n, r, inner], b [n, outer, r], scale fp32 [n], out
    and base [T, outer]; base may be out, and None stands for zeros.  a and b have x's type, or any
    type beside fp32 activations.  A call of many rows needs a workspace: the caller's (any contiguous
    tensor of enough bytes, 16-byte aligned) or one of its own,
    with room for copies where rows do not start at multiples of 16 bytes.  Many rows are faster with an a and
    b that start at such multiples too.
    """
    lib = gpu_lib()
    (dtype, gpu), T = _type("x", x), _dims("x", x, 2)[0]
    n, r, inner, outer, pa, pb, wtype = _adapter_shapes(a, b, gpu)
    px, ldx = _matrix("x", x, T, inner, x.dtype, gpu)
    po, ldo = _matrix("out", out, T, outer, x.dtype, gpu)
    p_base, ldb = (None, outer) if base is None else _matrix("base", base, T, outer, x.dtype, gpu)
    p_ad = _array("adapter", adapter, (T,), torch.int32, gpu)
    p_scale = _array("scale", scale, (n,), torch.float32, gpu)
    strided = (px | po | (p_base or 0) | (ldx | ldo | ldb) * x.element_size()) & 15
    need = _needed("moe_adapters_forward_workspace_strided" if strided and workspace is None else
                   "moe_adapters_forward_workspace", T, inner, outer, n, r)
    ws = _workspace(need, workspace, gpu, stream) if need else None
    _call(lib.moe_adapters_forward, (out,), gpu, stream, px, ldx, p_base, ldb, dtype, T, inner, outer, p_ad, pa, pb,
          wtype, p_scale, n, r, po, ldo, ws.data_ptr() if need else None, ws.numel() * ws.element_size() if need else 0)


def adapters_backward(d_out, x, adapter, a, b, scale, d_x, d_a, d_b, dx_base=None, workspace=None, stream=None):
    """Gradients of adapters_forward (moe_adapters_backward): d_x [T, inner] = dx_base + scale A_e^T B_e^T
    d_out, and the fp32 gradients d_a [n, r, inner] and d_b [n, outer, r] of all adapters.  dx_base may
    be d_x, and None stands for zeros; a workspace (any contiguous tensor of enough bytes, 16-byte
    aligned) may be kept by the caller."""
    lib = gpu_lib()
    (dtype, gpu), T = _type("x", x), _dims("x", x, 2)[0]
    n, r, inner, outer, pa, pb, wtype = _adapter_shapes(a, b, gpu)
    px, ldx = _matrix("x", x, T, inner, x.dtype, gpu)
    pd, ldd = _matrix("d_out", d_out, T, outer, x.dtype, gpu)
    pg, ldg = _matrix("d_x", d_x, T, inner, x.dtype, gpu)
    p_base, ldb = (None, inner) if dx_base is None else _matrix("dx_base", dx_base, T, inner, x.dtype, gpu)
    p_ad = _array("adapter", adapter, (T,), torch.int32, gpu)
    p_scale = _array("scale", scale, (n,), torch.float32, gpu)
    p_da = _array("d_a", d_a, (n, r, inner), torch.float32, gpu)
    p_db = _array("d_b", d_b, (n, outer, r), torch.float32, gpu)
    strided = (px | pd | pg | (p_base or 0) | (ldx | ldd | ldg | ldb) * x.element_size()) & 15
    need = _needed("moe_adapters_workspace_strided" if strided else "moe_adapters_workspace", T, inner, outer, n, r)
    ws = _workspace(need, workspace, gpu, stream)
    _call(lib.moe_adapters_backward, (d_x, d_a, d_b), gpu, stream, pd, ldd, px, ldx, p_base, ldb, dtype, T, inner, outer,
          p_ad, pa, pb, wtype, p_scale, n, r, pg, ldg, p_da, p_db, ws.data_ptr(), ws.numel() * ws.element_size())
