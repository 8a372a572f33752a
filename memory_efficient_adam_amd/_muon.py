"""ctypes marshalling for the Muon calls of libadam_mi355x.so (names follow
include/muon_mi355x.h)."""
import ctypes
import functools
import math

from . import _binding as B
from ._binding import ADAM_BLOCK_SIZE, AdamError, _check, _on, _stream, adam_last_error

MUON_STORAGES = {"bf16": 1, "q8": 2, "f32": 3}
MUON_SCALES = {"none": 0, "spectral": 1, "rms": 2}
MUON_MAX_STEPS = 16
_F_NESTEROV, _F_STOCHASTIC = 1, 2


class muon_layout(ctypes.Structure):
    _fields_ = [("storage", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("options", ctypes.c_uint32)]


class muon_iteration(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("eps", ctypes.c_float),
                ("coefficients", ctypes.POINTER(ctypes.c_float))]


class muon_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("scale", ctypes.c_int32),
                ("t", ctypes.c_int64), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("seed", ctypes.c_uint64), ("iteration", muon_iteration)]


class muon_matrices(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("batch", "rows", "cols", "x_batch_stride", "x_row_stride", "out_batch_stride",
                 "out_row_stride")] + [("x_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


_bound = None


def library():
    """The library with the Muon calls' signatures; raises if it is not built."""
    global _bound
    L = B.library()
    if _bound is L:
        return L
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    i64p, lay = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(muon_layout)
    signatures = {
        "muon_state_bytes": (i64, [i32, i64p, i64p, lay]),
        "muon_state_workspace_bytes": (i64, [i32, i64p, i64p, lay]),
        "muon_state_create": (i32, [ctypes.POINTER(vp), i32, i64p, i64p, lay, vp]),
        "muon_step": (i32, [vp, vp, vp, ctypes.POINTER(muon_hparams), lay, vp]),
        "muon_state_buffer_bytes": (i64, [vp, i32]),
        "muon_state_read": (i32, [vp, i32, vp, i64, vp]),
        "muon_state_write": (i32, [vp, i32, vp, i64, vp]),
        "muon_state_momentum": (i32, [vp, vp, i64, vp]),
        "muon_state_serialized_bytes": (i64, [vp]),
        "muon_state_save": (i32, [vp, vp, i64, vp]),
        "muon_state_load": (i32, [ctypes.POINTER(vp), vp, i64, vp]),
        "muon_state_set_draw_index": (i32, [vp, i64p, vp]),
        "muon_state_get_draw_index": (i32, [vp, i64p, i32]),
        "muon_state_describe": (i32, [vp, lay, i64p, i64p, i32]),
        "muon_state_destroy": (None, [vp]),
        "muon_orthogonalize_workspace_bytes": (i64, [i64, i64, i64]),
        "muon_orthogonalize": (i32, [ctypes.POINTER(muon_matrices), vp, vp,
                                     ctypes.POINTER(muon_iteration), vp, i64, vp]),
    }
    for name, (result, arguments) in signatures.items():
        f = getattr(L, name)
        f.restype, f.argtypes = result, arguments
    _bound = L
    return L


def _size(n):
    if n < 0:
        raise AdamError(int(n), adam_last_error())
    return int(n)


def _layout(storage, grad_dtype, block_size=ADAM_BLOCK_SIZE, options=0):
    return muon_layout(MUON_STORAGES.get(storage, storage) if isinstance(storage, str) else storage,
                       B.GRAD_DTYPES.get(grad_dtype, grad_dtype) if isinstance(grad_dtype, str)
                       else grad_dtype, block_size, options)


def _shapes(shapes):
    shapes = [(int(r), int(c)) for r, c in shapes]
    n = max(len(shapes), 1)
    return (shapes, (ctypes.c_int64 * n)(*[r for r, _ in shapes]),
            (ctypes.c_int64 * n)(*[c for _, c in shapes]))


def _iteration(steps, coefficients, eps):
    """coefficients: None (the default triple), one triple for every iteration, or
    one triple per iteration.  The struct keeps the array alive."""
    if coefficients is not None:
        coefficients = tuple(tuple(c) if isinstance(c, (tuple, list)) else c for c in coefficients)
    return _iteration_of(int(steps), coefficients, float(eps))


@functools.lru_cache(maxsize=64)
def _iteration_of(steps, coefficients, eps):
    values = None
    if coefficients is not None:
        rows = coefficients
        if len(rows) == 3 and all(isinstance(v, (int, float)) for v in rows):
            rows = [rows] * max(steps, 0)
        if len(rows) != steps or any(not isinstance(r, tuple) or len(r) != 3 for r in rows):
            raise ValueError(f"coefficients: expected three numbers or {steps} triples")
        if 0 < steps <= MUON_MAX_STEPS:  # other counts are the library's to refuse
            values = (ctypes.c_float * (3 * steps))(*[float(v) for r in rows for v in r])
    return muon_iteration(steps, eps, values)


def muon_state_bytes(shapes, storage, grad_dtype="f32", block_size=ADAM_BLOCK_SIZE):
    shapes, rows, cols = _shapes(shapes)
    lay = _layout(storage, grad_dtype, block_size)
    return _size(library().muon_state_bytes(len(shapes), rows, cols, ctypes.byref(lay)))


def muon_state_workspace_bytes(shapes, storage, grad_dtype="f32", block_size=ADAM_BLOCK_SIZE):
    shapes, rows, cols = _shapes(shapes)
    lay = _layout(storage, grad_dtype, block_size)
    return _size(library().muon_state_workspace_bytes(len(shapes), rows, cols, ctypes.byref(lay)))


class MuonState:
    """Owns one library state (freed on destroy() or garbage collection; after a
    graph capture, if that happens during one).
    device: the CUDA device index the state lives on (None: not recorded)."""

    def __init__(self, handle, shapes, layout, device=None):
        self.handle = handle
        self._set_shapes(shapes)
        self.layout = layout
        self.device = device
        # held here: globals may be gone when a state is collected at exit
        self._free, self._release = (library().muon_state_destroy, B._release) if handle else (None, None)
        B._release()
        self._checked = []  # tensor sets (held) and pointers of recent checked muon_step calls

    def _set_shapes(self, shapes):
        self.shapes = [tuple(s) for s in shapes]
        self.numels = [r * c for r, c in self.shapes]
        # each matrix's first entry in the padded flat state, and its length
        self.firsts, self.padded = [], 0
        for n in self.numels:
            self.firsts.append(self.padded)
            self.padded += -(-n // 16) * 16

    def __del__(self):
        self.destroy()

    def destroy(self):
        self._checked = []
        if getattr(self, "handle", None):
            handle, self.handle = self.handle, None
            self._release(self._free, handle)

    @property
    def storage(self):
        return {v: k for k, v in MUON_STORAGES.items()}[self.layout.storage]


def muon_state_create(shapes, storage, grad_dtype="f32", block_size=ADAM_BLOCK_SIZE, stream=None):
    """A state with zero momentum for matrices of the given (rows, cols) shapes:
    storage "f32", "bf16" or "q8" (8-bit codes with a scale per 2048 elements)."""
    shapes, rows, cols = _shapes(shapes)
    lay = _layout(storage, grad_dtype, block_size)
    h = ctypes.c_void_p()
    _check(library().muon_state_create(ctypes.byref(h), len(shapes), rows, cols, ctypes.byref(lay),
                                       _stream(stream)))
    return MuonState(h.value, shapes, lay, B._current_device())


def muon_state_destroy(state):
    state.destroy()


def _check_matrices(state, params, grads):
    if len(params) == len(grads) == len(state.shapes):
        for k, (p, g, shape) in enumerate(zip(params, grads, state.shapes)):
            for t in (p, g):
                if getattr(t, "shape", None) is not None and t.numel() == shape[0] * shape[1] and t.shape != shape:
                    raise ValueError(f"tensor {k}: param/grad shape {tuple(t.shape)}, the state "
                                     f"holds {shape}")
    B._check_step_tensors(state, params, grads)


def _launching_stream(stream):
    """The stream, which has to be one of the current device: kernels run on the
    stream's device, the pointers are this one's."""
    device = getattr(stream, "device", None)  # None, and raw handles, have none
    if device is not None and device.index != B._current_device():
        raise ValueError(f"the stream is on {device}, the current device is cuda:{B._current_device()}")
    return stream


def _form(tensors):
    """What a tensor can change (by .data, t_(), resize_()) while it stays the same object
    at the same address.  0.35 us a tensor."""
    return [(t.shape, t.dtype, t.is_contiguous()) for t in tensors]


def muon_step(state, params, grads, *, lr, t, momentum=0.95, weight_decay=0.0, nesterov=True,
              steps=5, coefficients=None, eps=1e-7, scale="rms", stochastic=False, seed=42,
              stream=None, expect=None):
    """One Muon step over all matrices: momentum, its orthogonalisation by
    `steps` Newton-Schulz iterations, p = p (1 - lr wd) - lr s O.  params: fp32
    device matrices (updated in place); grads: fp32 or bf16 ones.  scale: the
    factor s ("none", "spectral", "rms").  coefficients: a triple, or one per
    iteration.  expect: (storage, grad_dtype[, block_size[, options]]) the
    caller believes the state has."""
    P, G = B._checked_pointers(state, params, grads, _check_matrices, _form)
    if isinstance(scale, str) and scale not in MUON_SCALES:
        raise ValueError(f"scale must be one of {sorted(MUON_SCALES)}, got {scale!r}")
    hp = muon_hparams(lr, momentum, weight_decay,
                      MUON_SCALES[scale] if isinstance(scale, str) else int(scale), int(t),
                      (_F_NESTEROV if nesterov else 0) | (_F_STOCHASTIC if stochastic else 0), 0,
                      int(seed), _iteration(steps, coefficients, eps))
    lay = state.layout if expect is None else _layout(*expect)
    _check(library().muon_step(state.handle, ctypes.cast(P, ctypes.c_void_p),
                               ctypes.cast(G, ctypes.c_void_p), ctypes.byref(hp),
                               ctypes.byref(lay), _stream(_launching_stream(stream))))


def muon_state_buffer_bytes(state, which):
    w = B.BUFFERS.get(which, which) if isinstance(which, str) else which
    return _size(library().muon_state_buffer_bytes(state.handle, w))


def _exact_bytes(name, tensor, nbytes):
    if tensor.numel() * tensor.element_size() != nbytes or not tensor.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of exactly {nbytes} bytes, got "
                         f"{tensor.numel() * tensor.element_size()} bytes")


def muon_state_read(state, which, out=None, stream=None):
    """Copy a state buffer ("m_f32", "m_bf16", "m_codes", "m_scale") into a (new,
    device) torch tensor; bf16 momentum comes back as int16 bit patterns."""
    import torch
    nbytes = muon_state_buffer_bytes(state, which)
    if out is None:
        dt = getattr(torch, B._BUF_DTYPES[which])
        with _on(stream):
            out = torch.empty(nbytes // dt.itemsize, dtype=dt, device="cuda")
    _exact_bytes("out", out, nbytes)
    _check(library().muon_state_read(state.handle, B.BUFFERS[which], out.data_ptr(), nbytes,
                                     _stream(stream)))
    return out


def muon_state_write(state, which, src, stream=None):
    nbytes = muon_state_buffer_bytes(state, which)
    _exact_bytes("src", src, nbytes)
    _check(library().muon_state_write(state.handle, B.BUFFERS[which], src.data_ptr(), nbytes,
                                      _stream(stream)))


def muon_state_momentum(state, stream=None):
    """The momentum's values, one (rows, cols) tensor per matrix: fp32 (8-bit codes
    times their scale), or bf16 for bf16 storage.  A copy, in one allocation."""
    import torch
    with _on(stream):
        flat = torch.empty(state.padded, device="cuda",
                           dtype=torch.bfloat16 if state.layout.storage == 1 else torch.float32)
        _check(library().muon_state_momentum(state.handle, flat.data_ptr(),
                                             flat.numel() * flat.element_size(), _stream(None)))
    return [flat.as_strided(shape, (shape[1], 1), first) for shape, first in
            zip(state.shapes, state.firsts)]


def muon_state_describe(state):
    """(layout, shapes) of a state, as the library holds them."""
    lay = muon_layout()
    n = _size(library().muon_state_describe(state.handle, ctypes.byref(lay), None, None, 0))
    rows, cols = ((ctypes.c_int64 * max(n, 1))() for _ in range(2))
    library().muon_state_describe(state.handle, ctypes.byref(lay), rows, cols, n)
    return lay, [(int(rows[i]), int(cols[i])) for i in range(n)]


def muon_state_set_draw_index(state, first_index, stream=None):
    """Per matrix: the stochastic-rounding draw index of element 0."""
    n, arr = B._numels(first_index)
    if n != len(state.numels):
        raise ValueError(f"expected {len(state.numels)} draw indices")
    _check(library().muon_state_set_draw_index(state.handle, arr, _stream(stream)))


def muon_state_get_draw_index(state):
    n = len(state.numels)
    arr = (ctypes.c_int64 * max(n, 1))()
    _size(library().muon_state_get_draw_index(state.handle, arr, n))
    return [int(arr[i]) for i in range(n)]


def muon_state_serialized_bytes(state):
    return _size(library().muon_state_serialized_bytes(state.handle))


def muon_state_save(state, stream=None):
    """The serialized state as a numpy uint8 array (host memory)."""
    import numpy as np
    out = np.empty(muon_state_serialized_bytes(state), np.uint8)
    _check(library().muon_state_save(state.handle, out.ctypes.data, out.size, _stream(stream)))
    return out


def muon_state_load(buf, stream=None):
    """A new state holding the contents of a serialized state (bytes-like or
    numpy uint8 array)."""
    import numpy as np
    arr = np.ascontiguousarray(np.frombuffer(buf, np.uint8) if not isinstance(buf, np.ndarray)
                               else buf.view(np.uint8))
    h = ctypes.c_void_p()
    _check(library().muon_state_load(ctypes.byref(h), arr.ctypes.data, arr.size, _stream(stream)))
    st = MuonState(h.value, [], muon_layout(), B._current_device())
    st.layout, shapes = muon_state_describe(st)
    st._set_shapes(shapes)
    return st


# ---------------------------------------------------------------- orthogonalisation
def _has_tangent(t):
    """Whether t is a dual tensor of the forward-mode level that is open, if one is."""
    from torch.autograd import forward_ad
    return forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None


_DTYPE_CODES = {"torch.float32": 0, "torch.bfloat16": 1}


@functools.lru_cache(maxsize=256)
def _matrices_of(name, shape, stride, dtype):
    """(batch, rows, cols, batch stride, row stride, dtype code) of a tensor of
    matrices whose rows are contiguous and whose batch has one stride."""
    code = _DTYPE_CODES.get(str(dtype))
    if code is None:
        raise ValueError(f"{name}: dtype {dtype}, expected torch.float32 or torch.bfloat16")
    if len(shape) < 2:
        raise ValueError(f"{name}: expected (..., rows, cols), got {shape}")
    rows, cols = shape[-2:]
    if 0 in shape:  # nothing to read: any strides will do
        return math.prod(shape[:-2]), rows, cols, rows * cols, cols, code
    batch, batch_stride = 1, 0
    for n, s in zip(reversed(shape[:-2]), reversed(stride[:-2])):
        if n == 1:
            continue
        if batch != 1 and s != batch * batch_stride:
            raise ValueError(f"{name}: the batch dimensions must have one stride between matrices")
        if batch == 1:
            batch_stride = s
        batch *= n
    row_stride = stride[-2] if rows > 1 else cols
    if cols > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    if row_stride < cols:
        raise ValueError(f"{name}: rows overlap")
    return batch, rows, cols, batch_stride, row_stride, code


@functools.lru_cache(maxsize=256)
def muon_orthogonalize_workspace_bytes(batch, rows, cols):
    return _size(library().muon_orthogonalize_workspace_bytes(batch, rows, cols))


def muon_orthogonalize(x, *, out=None, steps=5, coefficients=None, eps=1e-7, workspace=None,
                       stream=None):
    """The Newton-Schulz orthogonalisation of each matrix of x (..., rows, cols),
    fp32 or bf16, rows contiguous, one stride between matrices.  out: of x's shape,
    fp32 or bf16 (default: a new tensor of x's type; x itself for in place).
    workspace: a contiguous device tensor of at least
    muon_orthogonalize_workspace_bytes bytes that calls ordered on one stream may
    share (default: allocated for the call).  No gradient is defined through it,
    backward or forward: tensors that ask for one are refused."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch tensor")
    batch, rows, cols, x_batch, x_row, x_code = _matrices_of("x", tuple(x.shape), x.stride(), x.dtype)
    if out is not None and (not isinstance(out, torch.Tensor) or out.shape != x.shape):
        raise ValueError("out must be a tensor of x's shape")
    if torch.is_grad_enabled() and (x.requires_grad or (out is not None and out.requires_grad)):
        raise ValueError("no gradient is defined through muon_orthogonalize: detach its input or "
                         "call it under torch.no_grad()")
    if _has_tangent(x) or (out is not None and _has_tangent(out)):
        raise ValueError("no forward-mode gradient is defined through muon_orthogonalize: pass the "
                         "primal of a dual tensor")
    it = _iteration(steps, coefficients, eps)
    for name, t in (("x", x), ("out", out), ("workspace", workspace)):
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA (HIP) device tensor")
        if t.get_device() != B._current_device():
            raise ValueError(f"{name} is on {t.device}, the current device is "
                             f"cuda:{B._current_device()}")
        if t is workspace and not t.is_contiguous():
            raise ValueError("workspace must be contiguous")
    need = muon_orthogonalize_workspace_bytes(batch, rows, cols)
    with _on(_launching_stream(stream)):
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        at, nbytes = ((0, 0) if workspace is None else
                      (workspace.data_ptr(), workspace.numel() * workspace.element_size()))
        _, _, _, out_batch, out_row, out_code = _matrices_of("out", tuple(out.shape), out.stride(),
                                                             out.dtype)
        mats = muon_matrices(batch, rows, cols, x_batch, x_row, out_batch, out_row, x_code, out_code)
        _check(library().muon_orthogonalize(ctypes.byref(mats), x.data_ptr(), out.data_ptr(),
                                            ctypes.byref(it), at, nbytes, _stream(None)))
    return out
