"""ctypes marshalling for the embedding calls of libadam_mi355x.so (names follow
include/embedding_mi355x.h).

The calls on few tokens take some 4 us on the GPU, so what a call derives from its
tensors' sizes, strides and types (the C call's shape, its checks, the workspace's
size) is remembered by exactly those, in _lookup_form and _gradient_form."""
import ctypes
import functools
import math

from . import _binding as B
from ._binding import AdamError, _check, _on, adam_last_error
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


def _check_tensors(*named):
    """Tensors of the current device, as (name, tensor) pairs (None: not given)."""
    import torch
    current = B._current_device()
    for name, t in named:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA (HIP) device tensor")
        if t.get_device() != current:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{current}")


def _check_no_gradient(what, *named):
    import torch
    for name, t in named:
        if t is None:
            continue
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"no gradient is defined through {what}: detach {name} or call it under torch.no_grad()")
        if _has_tangent(t):
            raise ValueError(f"no forward-mode gradient is defined through {what}: pass the primal of {name}")


def _current_stream(device):
    import torch
    return torch._C._cuda_getCurrentRawStream(device)


def _written(tensor):
    """Counts a tensor that the library wrote as torch counts one written in place, so that a graph which
    kept its old values raises in its backward pass.  (0.5 us)"""
    import torch
    torch._C._increment_version([tensor])


# ---------------------------------------------------------------- lookup
def _signed(scale):
    """scale as a key: 0.0 and -0.0 are equal, but not what they make of a value."""
    return scale, math.copysign(1.0, scale)


@functools.lru_cache(maxsize=512)
def _lookup_form(table_shape, table_stride, table_dtype, token_shape, token_dtype, out_shape, out_stride, out_dtype, scale):
    """The C call's shape.  out_stride: None for a new tensor's; scale: as _signed has it."""
    if len(table_shape) != 2:
        raise ValueError(f"table: expected (rows, cols), got {tuple(table_shape)}")
    rows, cols = table_shape
    want = tuple(token_shape) + (cols,)
    if out_stride is not None and tuple(out_shape) != want:
        raise ValueError(f"out must have the shape {want} and, if one is given, dtype")
    count = 1
    for n in token_shape:
        count *= n
    return embedding_shape(rows, cols, count, _row_stride("table", table_shape, table_stride),
                           cols if out_stride is None else _row_stride("out", out_shape, out_stride),
                           _dtype("table", table_dtype), _dtype("dtype", out_dtype),
                           _dtype("tokens", token_dtype, _TOKEN_DTYPES), scale[0])


def _lookup(table, tokens, scale, dtype, out):
    import torch
    given = out is not None
    if not given:
        shape = _lookup_form(table.shape, table.stride(), table.dtype, tokens.shape, tokens.dtype, None, None, dtype,
                             _signed(scale))
        out = torch.empty((*tokens.shape, table.shape[1]), dtype=dtype, device=table.device)
    else:
        shape = _lookup_form(table.shape, table.stride(), table.dtype, tokens.shape, tokens.dtype, out.shape, out.stride(),
                             dtype, _signed(scale))
    tokens = tokens.contiguous()
    _check(library().embedding_lookup(shape, table.data_ptr(), tokens.data_ptr(), out.data_ptr(),
                                      _current_stream(table.get_device())))
    if given:
        _written(out)
    return out


@functools.lru_cache(maxsize=1)
def _function():
    import torch
    from torch.autograd.function import once_differentiable

    class Lookup(torch.autograd.Function):
        @staticmethod
        def forward(ctx, table, tokens, scale, dtype):
            ctx.save_for_backward(tokens)
            ctx.rows, ctx.scale, ctx.dtype = table.shape[0], scale, table.dtype
            return _lookup(table, tokens, scale, dtype, None)

        @staticmethod
        @once_differentiable
        def backward(ctx, grad):
            if torch.cuda.is_current_stream_capturing():
                raise ValueError("the backward pass of an eager lookup cannot be captured: record embedding_gradient")
            tokens, = ctx.saved_tensors
            return embedding_gradient(grad.contiguous(), tokens, ctx.rows, scale=ctx.scale,
                                      dtype=ctx.dtype), None, None, None
    return Lookup


def embedding_lookup(table, tokens, *, scale=1.0, dtype=None, out=None, stream=None):
    """scale * table[tokens], rows of zeros for tokens outside the table
    (padding).  table: (rows, cols), fp32 or bf16, rows contiguous; tokens: int32 or
    int64, any shape.  dtype: the result's (default: the table's).  out: a
    tensor of tokens' shape + (cols,) to write instead of a new one.  If the table asks for
    a gradient it gets the dense one of embedding_gradient (in a backward pass; not in forward
    mode, and with no out).  Neither that lookup nor its backward pass can be captured into a graph:
    a leaf's gradient is summed on the stream of the eager graph that first asked for it, and while such a graph lives
    a capture that meets it ends the process, which cannot be seen from here.  A captured step
    records embedding_lookup under torch.no_grad(), and embedding_gradient or embedding_adam_step."""
    import torch
    _check_tensors(("table", table), ("tokens", tokens), ("out", out))
    if out is not None and dtype not in (None, out.dtype):
        raise ValueError(f"out has dtype {out.dtype}, not {dtype}")
    dtype = out.dtype if out is not None else dtype or table.dtype
    if _has_tangent(table):
        raise ValueError("no forward-mode gradient is defined through embedding_lookup: pass the primal of table")
    _launching_stream(stream)
    if (table.requires_grad or (out is not None and out.requires_grad)) and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("no gradient is defined through out: detach table and out, or call it under torch.no_grad()")
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("a lookup with a gradient cannot be captured: record embedding_lookup under "
                             "torch.no_grad(), and embedding_gradient")
        with _on(stream):
            return _function().apply(table, tokens, float(scale), dtype)
    if stream is None:
        return _lookup(table, tokens, float(scale), dtype, out)
    with _on(stream):
        return _lookup(table, tokens, float(scale), dtype, out)


# ---------------------------------------------------------------- gradient
@functools.lru_cache(maxsize=512)
def embedding_gradient_workspace_bytes(tokens, rows, cols):
    n = library().embedding_gradient_workspace_bytes(tokens, rows, cols)
    if n < 0:
        raise AdamError(int(n), adam_last_error())
    return int(n)


@functools.lru_cache(maxsize=512)
def _gradient_form(grad_shape, grad_stride, grad_dtype, token_shape, token_dtype, rows, out_shape, out_stride, out_dtype,
                   scale):
    """The C call's shape and the bytes of its workspace.  out_stride: None for a new
    tensor's; scale: as _signed has it."""
    if len(grad_shape) != len(token_shape) + 1 or grad_shape[:-1] != token_shape:
        raise ValueError(f"grad must have tokens' shape and one dimension more, got {tuple(grad_shape)} for "
                         f"{tuple(token_shape)}")
    cols = grad_shape[-1]
    if out_stride is not None and tuple(out_shape) != (rows, cols):
        raise ValueError(f"out must have the shape {(rows, cols)} and, if one is given, dtype")
    count = 1
    for n in token_shape:
        count *= n
    shape = embedding_shape(rows, cols, count, cols if out_stride is None else _row_stride("out", out_shape, out_stride),
                            _row_stride("grad", grad_shape, grad_stride), _dtype("dtype", out_dtype),
                            _dtype("grad", grad_dtype), _dtype("tokens", token_dtype, _TOKEN_DTYPES), scale[0])
    return shape, embedding_gradient_workspace_bytes(count, rows, cols)


def _workspace(workspace, need, device):
    """What holds the workspace of a call on the current stream, and its bytes."""
    import torch
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device), need
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


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
    _check_tensors(("grad", grad), ("tokens", tokens), ("out", out), ("workspace", workspace))
    _check_no_gradient("embedding_gradient", ("grad", grad), ("out", out))
    rows = int(rows)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        if rows < 0:
            raise ValueError(f"rows must not be negative, got {rows}")
        dtype = dtype or torch.float32
        form = _gradient_form(grad.shape, grad.stride(), grad.dtype, tokens.shape, tokens.dtype, rows, None, None, dtype,
                              _signed(float(scale)))
    else:
        if dtype not in (None, out.dtype):
            raise ValueError(f"out has dtype {out.dtype}, not {dtype}")
        form = _gradient_form(grad.shape, grad.stride(), grad.dtype, tokens.shape, tokens.dtype, rows, out.shape,
                              out.stride(), out.dtype, _signed(float(scale)))
    shape, need = form
    given = out is not None
    with _on(_launching_stream(stream)):
        tokens = tokens.contiguous()
        if not given:
            out = torch.empty((rows, grad.shape[-1]), dtype=dtype, device=grad.device)
        workspace, nbytes = _workspace(workspace, need, grad.device)
        _check(library().embedding_gradient(shape, grad.data_ptr(), tokens.data_ptr(), out.data_ptr(),
                                            1 if accumulate else 0, workspace.data_ptr(), nbytes,
                                            _current_stream(grad.get_device())))
    if given:
        _written(out)
    return out


# ---------------------------------------------------------------- step
@functools.lru_cache(maxsize=64)
def _buffer_sizes(numel, amsgrad):
    return B.state_buffer_sizes([numel], "f32", amsgrad)


def embedding_adam_step(table, grad, tokens, buffers, *, amsgrad=False, scale=1.0, lr, beta1, beta2, eps, weight_decay,
                        t, decoupled=True, workspace=None, stream=None):
    """The Adam/AdamW step with fp32 moments on the rows of table that tokens name, its
    gradient taken from grad and tokens as embedding_gradient takes it; other rows
    and their state stay as they are.  table: (rows, cols), fp32, contiguous, updated in
    place.  buffers: the caller-owned state of adam_step_noalloc for this one tensor
    (state_buffer_sizes([rows * cols], "f32", amsgrad); zeros for a new state), on which
    either kind of step may be taken."""
    import torch
    _check_tensors(("table", table), ("grad", grad), ("tokens", tokens), ("workspace", workspace))
    _check_no_gradient("embedding_adam_step", ("grad", grad))
    if table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous():
        raise ValueError("table must be a contiguous fp32 tensor (rows, cols)")
    rows, cols = table.shape
    if grad.dim() == 0 or grad.shape[-1] != cols:
        raise ValueError(f"grad must have {cols} columns as the table has, got {tuple(grad.shape)}")
    shape, need = _gradient_form(grad.shape, grad.stride(), grad.dtype, tokens.shape, tokens.dtype, rows, table.shape,
                                 (cols, 1), table.dtype, _signed(float(scale)))
    want = _buffer_sizes(rows * cols, bool(amsgrad))
    if buffers.keys() != want.keys():
        raise ValueError(f"buffers must be exactly {sorted(want)}, got {sorted(buffers)}")
    state = (ctypes.c_void_p * len(B.BUFFERS))()
    _check_tensors(*[("buffer " + name, buffers[name]) for name in want])
    for name, nbytes in want.items():
        b = buffers[name]
        if b.numel() * b.element_size() != nbytes or not b.is_contiguous():
            raise ValueError(f"buffer {name}: must be a contiguous tensor of {nbytes} bytes")
        state[B.BUFFERS[name]] = b.data_ptr()
    hp = B._hparams(lr, beta1, beta2, eps, weight_decay, t, decoupled, False, None, 0, False)
    layout = B.adam_layout(B.STORAGES["f32"], shape.value_dtype, B.ADAM_BLOCK_SIZE, B.OPT_AMSGRAD if amsgrad else 0)
    with _on(_launching_stream(stream)):
        tokens = tokens.contiguous()
        workspace, nbytes = _workspace(workspace, need, table.device)
        _check(library().embedding_adam_step(shape, table.data_ptr(), grad.data_ptr(), tokens.data_ptr(),
                                             ctypes.addressof(state), hp, layout, workspace.data_ptr(), nbytes,
                                             _current_stream(table.get_device())))
    _written(table)
