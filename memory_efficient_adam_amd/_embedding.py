"""ctypes marshalling for the embedding calls of libadam_mi355x.so (names follow
include/embedding_mi355x.h)."""
import ctypes
import functools

from . import _binding as B
from ._binding import AdamError, _check, _on, _stream, adam_last_error
from ._muon import _has_tangent, _launching_stream


class embedding_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "cols", "tokens", "table_stride", "value_stride")] + \
               [(n, ctypes.c_int32) for n in ("table_dtype", "value_dtype", "token_dtype")] + \
               [("scale", ctypes.c_float)]


_bound = None


def library():
    """The library with the embedding calls' signatures; raises if it is not built."""
    global _bound
    L = B.library()
    if _bound is L:
        return L
    vp, i64, i32, shape = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.POINTER(embedding_shape)
    signatures = {
        "embedding_lookup": (i32, [shape, vp, vp, vp, vp]),
        "embedding_gradient_workspace_bytes": (i64, [i64, i64, i64]),
        "embedding_gradient": (i32, [shape, vp, vp, vp, i32, vp, i64, vp]),
        "embedding_adam_step": (i32, [shape, vp, vp, vp, vp, ctypes.POINTER(B.adam_hparams),
                                      ctypes.POINTER(B.adam_layout), vp, i64, vp]),
    }
    for name, (result, arguments) in signatures.items():
        f = getattr(L, name)
        f.restype, f.argtypes = result, arguments
    _bound = L
    return L


_DTYPES = {"torch.float32": 0, "torch.bfloat16": 1}
_TOKEN_DTYPES = {"torch.int32": 0, "torch.int64": 1}


def _dtype(name, dtype, codes=_DTYPES):
    code = codes.get(str(dtype))
    if code is None:
        raise ValueError(f"{name}: dtype {dtype}, expected one of {', '.join(codes)}")
    return code


@functools.lru_cache(maxsize=256)
def _row_stride(name, shape, stride):
    """Elements between the rows of a tensor (.., cols) whose rows are contiguous
    and whose other dimensions have one stride between rows."""
    if 0 in shape:  # nothing to read: any strides will do
        return shape[-1]
    if shape[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    count, between = 1, 0
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if count != 1 and s != count * between:
            raise ValueError(f"{name}: its rows must have one stride between them")
        if count == 1:
            between = s
        count *= n
    return between if count > 1 else shape[-1]


def _check_tensors(**tensors):
    """Tensors of the current device (None: not given)."""
    import torch
    current = B._current_device()
    for name, t in tensors.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA (HIP) device tensor")
        if t.get_device() != current:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{current}")


def _check_no_gradient(what, **tensors):
    import torch
    for name, t in tensors.items():
        if t is None:
            continue
        if torch.is_grad_enabled() and t.requires_grad:
            raise ValueError(f"no gradient is defined through {what}: detach {name} or call it under torch.no_grad()")
        if _has_tangent(t):
            raise ValueError(f"no forward-mode gradient is defined through {what}: pass the primal of {name}")


def _table_of(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected (rows, cols), got {tuple(t.shape)}")
    return _dtype(name, t.dtype), _row_stride(name, tuple(t.shape), t.stride())


def _shape_of(rows, cols, tokens, table_stride, value_stride, table_dtype, value_dtype, scale):
    return embedding_shape(rows, cols, tokens.numel(), table_stride, value_stride, table_dtype, value_dtype,
                           _dtype("tokens", tokens.dtype, _TOKEN_DTYPES), float(scale))


# ---------------------------------------------------------------- lookup
def _lookup(table, tokens, scale, dtype, out, stream):
    import torch
    rows, cols = table.shape
    table_code, table_stride = _table_of("table", table)
    with _on(_launching_stream(stream)):
        tokens = tokens.contiguous()
        if out is None:
            out = torch.empty(tokens.shape + (cols,), dtype=dtype, device=table.device)
        shape = _shape_of(rows, cols, tokens, table_stride, _row_stride("out", tuple(out.shape), out.stride()),
                          table_code, _dtype("out", out.dtype), scale)
        _check(library().embedding_lookup(ctypes.byref(shape), table.data_ptr(), tokens.data_ptr(), out.data_ptr(),
                                          _stream(None)))
    return out


@functools.lru_cache(maxsize=1)
def _function():
    import torch
    from torch.autograd.function import once_differentiable

    class Lookup(torch.autograd.Function):
        @staticmethod
        def forward(ctx, table, tokens, scale, dtype, stream):
            ctx.save_for_backward(tokens)
            ctx.rows, ctx.scale, ctx.dtype = table.shape[0], scale, table.dtype
            return _lookup(table, tokens, scale, dtype, None, stream)

        @staticmethod
        @once_differentiable
        def backward(ctx, grad):
            tokens, = ctx.saved_tensors
            return embedding_gradient(grad.contiguous(), tokens, ctx.rows, scale=ctx.scale,
                                      dtype=ctx.dtype), None, None, None, None
    return Lookup


def embedding_lookup(table, tokens, *, scale=1.0, dtype=None, out=None, stream=None):
    """scale * table[tokens], rows of zeros for tokens outside the table
    (padding).  table: (rows, cols), fp32 or bf16, rows contiguous; tokens: int32 or
    int64, any shape.  dtype: the result's (default: the table's).  out: a
    tensor of tokens' shape + (cols,) to write instead of a new one.  If the table asks for
    a gradient it gets the dense one of embedding_gradient (in a backward pass; in neither a
    graph capture nor forward mode, and with no out)."""
    import torch
    _check_tensors(table=table, tokens=tokens, out=out)
    _table_of("table", table)
    if out is not None and (out.shape != tokens.shape + table.shape[1:] or dtype not in (None, out.dtype)):
        raise ValueError(f"out must have the shape {tuple(tokens.shape + table.shape[1:])} and, if one is given, dtype")
    dtype = dtype or table.dtype
    _dtype("dtype", dtype)
    _dtype("tokens", tokens.dtype, _TOKEN_DTYPES)
    if _has_tangent(table):
        raise ValueError("no forward-mode gradient is defined through embedding_lookup: pass the primal of table")
    if torch.is_grad_enabled() and (table.requires_grad or (out is not None and out.requires_grad)):
        if out is not None:
            raise ValueError("no gradient is defined through out: detach table and out, or call it under torch.no_grad()")
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("a lookup with a gradient cannot be captured: record embedding_lookup under "
                             "torch.no_grad(), and embedding_gradient")
        _launching_stream(stream)
        with _on(stream):
            return _function().apply(table, tokens, scale, dtype, None)
    return _lookup(table, tokens, scale, dtype, out, stream)


# ---------------------------------------------------------------- gradient
@functools.lru_cache(maxsize=256)
def embedding_gradient_workspace_bytes(tokens, rows, cols):
    n = library().embedding_gradient_workspace_bytes(tokens, rows, cols)
    if n < 0:
        raise AdamError(int(n), adam_last_error())
    return int(n)


def _check_grad(grad, tokens):
    if grad.dim() != tokens.dim() + 1 or grad.shape[:-1] != tokens.shape:
        raise ValueError(f"grad must have tokens' shape and one dimension more, got {tuple(grad.shape)} for "
                         f"{tuple(tokens.shape)}")
    return _dtype("grad", grad.dtype), _row_stride("grad", tuple(grad.shape), grad.stride())


def _workspace(workspace, need, device):
    """(address, bytes, what holds it) of the workspace of a call on the current stream."""
    import torch
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def embedding_gradient(grad, tokens, rows, *, scale=1.0, dtype=None, out=None, accumulate=False, workspace=None,
                       stream=None):
    """The gradient of embedding_lookup's table of `rows` rows: for each row scale times
    the sum of grad's rows whose token it is.  grad: tokens' shape + (cols,), fp32 or bf16,
    rows contiguous, one stride between them; rows of padding are not read.  Written whole
    to out (default: a new tensor of dtype, itself fp32 by default), or with accumulate
    added to it.  workspace: a contiguous device tensor of at least
    embedding_gradient_workspace_bytes(tokens, rows, cols) bytes that calls ordered on
    one stream may share (default: allocated for the call)."""
    import torch
    _check_tensors(grad=grad, tokens=tokens, out=out, workspace=workspace)
    _check_no_gradient("embedding_gradient", grad=grad, out=out)
    code, stride = _check_grad(grad, tokens)
    rows, cols = int(rows), grad.shape[-1]
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        if rows < 0:
            raise ValueError(f"rows must not be negative, got {rows}")
        _dtype("dtype", dtype or torch.float32)
    elif tuple(out.shape) != (rows, cols) or dtype not in (None, out.dtype):
        raise ValueError(f"out must have the shape {(rows, cols)} and, if one is given, dtype")
    need = embedding_gradient_workspace_bytes(tokens.numel(), rows, cols)
    with _on(_launching_stream(stream)):
        tokens = tokens.contiguous()
        if out is None:
            out = torch.empty(rows, cols, dtype=dtype or torch.float32, device=grad.device)
        out_code, out_stride = _table_of("out", out)
        shape = _shape_of(rows, cols, tokens, out_stride, stride, out_code, code, scale)
        at, nbytes, _held = _workspace(workspace, need, grad.device)
        _check(library().embedding_gradient(ctypes.byref(shape), grad.data_ptr(), tokens.data_ptr(), out.data_ptr(),
                                            int(bool(accumulate)), at, nbytes, _stream(None)))
    return out


# ---------------------------------------------------------------- step
def embedding_adam_step(table, grad, tokens, buffers, *, amsgrad=False, scale=1.0, lr, beta1, beta2, eps, weight_decay,
                        t, decoupled=True, workspace=None, stream=None):
    """The Adam/AdamW step with fp32 moments on the rows of table that tokens name, its
    gradient taken from grad and tokens as embedding_gradient takes it; other rows
    and their state stay as they are.  table: (rows, cols), fp32, contiguous, updated in
    place.  buffers: the caller-owned state of adam_step_noalloc for this one tensor
    (state_buffer_sizes([rows * cols], "f32", amsgrad); zeros for a new state), on which
    either kind of step may be taken."""
    import torch
    _check_tensors(table=table, grad=grad, tokens=tokens, workspace=workspace)
    _check_no_gradient("embedding_adam_step", grad=grad)
    code, stride = _check_grad(grad, tokens)
    if table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous():
        raise ValueError("table must be a contiguous fp32 tensor (rows, cols)")
    rows, cols = table.shape
    if grad.shape[-1] != cols:
        raise ValueError(f"grad has {grad.shape[-1]} columns, the table {cols}")
    want = B.state_buffer_sizes([rows * cols], "f32", amsgrad)
    if set(buffers) != set(want):
        raise ValueError(f"buffers must be exactly {sorted(want)}, got {sorted(buffers)}")
    state = (ctypes.c_void_p * len(B.BUFFERS))()
    _check_tensors(**{f"buffer {name}": b for name, b in buffers.items()})
    for name, nbytes in want.items():
        b = buffers[name]
        if b.numel() * b.element_size() != nbytes or not b.is_contiguous():
            raise ValueError(f"buffer {name}: must be a contiguous tensor of {nbytes} bytes")
        state[B.BUFFERS[name]] = b.data_ptr()
    need = embedding_gradient_workspace_bytes(tokens.numel(), rows, cols)
    hp = B._hparams(lr, beta1, beta2, eps, weight_decay, t, decoupled, False, None, 0, False)
    layout = B._layout("f32", code, options=B.OPT_AMSGRAD if amsgrad else 0)
    with _on(_launching_stream(stream)):
        tokens = tokens.contiguous()
        shape = _shape_of(rows, cols, tokens, cols, stride, 0, code, scale)
        at, nbytes, _held = _workspace(workspace, need, table.device)
        _check(library().embedding_adam_step(ctypes.byref(shape), table.data_ptr(), grad.data_ptr(), tokens.data_ptr(),
                                             ctypes.cast(state, ctypes.c_void_p), ctypes.byref(hp),
                                             ctypes.byref(layout), at, nbytes, _stream(None)))
