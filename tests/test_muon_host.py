"""Host-side checks of the Muon calls that need no GPU: exports, struct
layouts, sizes against their closed forms, argument errors before any device
call, the checkpoint stream's validation, and the binding's tensor checks."""
import ctypes
import os
import re
import struct

import pytest
import torch

import memory_efficient_adam_amd as ma
from memory_efficient_adam_amd import _binding as B
from memory_efficient_adam_amd import _muon as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "muon_mi355x.h")
HP = dict(lr=1e-3, t=1)


def _arr(values):
    return (ctypes.c_int64 * max(len(values), 1))(*values)


def test_library_exports_every_declared_function():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(muon_[a-z_]+)\s*\(", src)))
    assert {"muon_step", "muon_orthogonalize", "muon_state_create"} <= set(names)
    lib = ctypes.CDLL(ma.library_path())
    for n in names:
        assert hasattr(lib, n), n
        assert hasattr(ma, n), n


def test_structs_match_the_header():
    assert ctypes.sizeof(M.muon_layout) == 16
    assert ctypes.sizeof(M.muon_iteration) == 16 and M.muon_iteration.coefficients.offset == 8
    assert ctypes.sizeof(M.muon_hparams) == 56
    assert M.muon_hparams.t.offset == 16 and M.muon_hparams.seed.offset == 32
    assert M.muon_hparams.iteration.offset == 40
    assert ctypes.sizeof(M.muon_matrices) == 64 and M.muon_matrices.x_dtype.offset == 56


@pytest.mark.parametrize("storage,e,s", [("f32", 4, 0), ("bf16", 2, 0), ("q8", 1, 4)])
def test_state_bytes_closed_form(storage, e, s):
    shapes = [(1, 1), (33, 65), (0, 7), (2048, 2), (100, 100)]
    want = sum((r * c + 15) // 16 * 16 * e + -(-r * c // 2048) * s for r, c in shapes)
    assert ma.muon_state_bytes(shapes, storage) == want
    assert ma.muon_state_bytes([], storage) == 0 == ma.muon_state_workspace_bytes([], storage)


def test_workspace_covers_the_factors():
    # four X arrays and five square ones of 4 bytes an element, at least
    for shapes in ([(1000, 768)], [(2304, 768)] * 12, [(4096, 4096)] * 4, [(65, 65)]):
        most = ma.muon_state_workspace_bytes(shapes, "f32")
        r, c = shapes[0]
        assert most >= 16 * r * c + 20 * min(r, c) ** 2
    one = ma.muon_state_workspace_bytes([(4096, 4096)] * 4, "f32")
    assert ma.muon_state_workspace_bytes([(4096, 4096)] * 400, "f32") == one  # a part at a time
    assert ma.muon_orthogonalize_workspace_bytes(1000, 64, 768) == 0
    assert ma.muon_orthogonalize_workspace_bytes(0, 1000, 768) == 0
    assert ma.muon_orthogonalize_workspace_bytes(1, 65, 768) >= 16 * 65 * 768 + 20 * 65 * 65


@pytest.mark.parametrize("shapes", [[(-1, 4)], [(4, -1)], [(2 ** 21, 1)], [(2 ** 20, 2 ** 13)]])
def test_bad_shapes_are_refused(shapes):
    for f in (ma.muon_state_bytes, ma.muon_state_workspace_bytes):
        with pytest.raises(ma.AdamError) as e:
            f(shapes, "q8")
        assert e.value.code == -1
    with pytest.raises(ma.AdamError):
        M.muon_orthogonalize_workspace_bytes(1, *shapes[0])


def test_bad_layouts_are_refused():
    lib = M.library()
    h = ctypes.c_void_p()
    for lay in (M._layout(9, "f32"), M._layout("q8", 7), M._layout("q8", "f32", 1024), M._layout("q8", "f32", 2048, 1)):
        assert lib.muon_state_bytes(1, _arr([4]), _arr([4]), ctypes.byref(lay)) == -1
        assert lib.muon_state_create(ctypes.byref(h), 1, _arr([4]), _arr([4]), ctypes.byref(lay), None) == -1
    good = M._layout("q8", "f32")
    assert lib.muon_state_create(None, 1, _arr([4]), _arr([4]), ctypes.byref(good), None) == -1
    assert lib.muon_state_create(ctypes.byref(h), 1, None, _arr([4]), ctypes.byref(good), None) == -1
    assert lib.muon_state_create(ctypes.byref(h), -1, None, None, ctypes.byref(good), None) == -1
    assert lib.muon_state_create(ctypes.byref(h), 1, _arr([4]), _arr([4]), None, None) == -1
    assert h.value is None
    assert "NULL" in ma.adam_last_error()  # one error text for the library


def test_null_states_are_refused():
    lib = M.library()
    hp, lay = M.muon_hparams(), M._layout("q8", "f32")
    assert lib.muon_step(None, None, None, ctypes.byref(hp), ctypes.byref(lay), None) == -1
    assert lib.muon_state_buffer_bytes(None, 0) == -1
    assert lib.muon_state_read(None, 0, None, 0, None) == -1
    assert lib.muon_state_write(None, 0, None, 0, None) == -1
    assert lib.muon_state_momentum(None, None, 0, None) == -1
    assert lib.muon_state_serialized_bytes(None) == -1
    assert lib.muon_state_save(None, None, 0, None) == -1
    assert lib.muon_state_set_draw_index(None, None, None) == -1
    assert lib.muon_state_get_draw_index(None, None, 0) == -1
    assert lib.muon_state_describe(None, None, None, None, 0) == -1
    lib.muon_state_destroy(None)


# ---------------------------------------------------------------- orthogonalisation arguments
# The pointers below are never dereferenced: every case ends at a host check.
X, OUT, WS = 1 << 30, 1 << 34, 1 << 38


def _orth(mats=None, it=None, x=X, out=OUT, ws=WS, ws_bytes=1 << 40, **over):
    m = dict(batch=2, rows=100, cols=80, x_batch_stride=8000, x_row_stride=80, out_batch_stride=8000,
             out_row_stride=80, x_dtype=0, out_dtype=0)
    m.update(over)
    mats = M.muon_matrices(*[m[n] for n, _ in M.muon_matrices._fields_]) if mats is None else mats
    it = M._iteration(5, None, 1e-7) if it is None else it
    return M.library().muon_orthogonalize(ctypes.byref(mats), x, out, ctypes.byref(it), ws, ws_bytes, None)


@pytest.mark.parametrize("what,kw,code", [
    ("batch", dict(batch=-1), -1), ("dimension", dict(rows=2 ** 21), -1), ("row stride", dict(x_row_stride=79), -1),
    ("row stride", dict(out_row_stride=0), -1), ("stride", dict(x_batch_stride=-1), -1),
    ("stride", dict(x_row_stride=2 ** 41), -1), ("dtype", dict(x_dtype=2), -1), ("dtype", dict(out_dtype=-1), -1),
    ("NULL", dict(x=0), -1), ("NULL", dict(out=0), -1), ("NULL", dict(ws=0), -1), ("needed", dict(ws_bytes=1000), -1),
    ("overlap", dict(out_batch_stride=7999), -1), ("overlaps", dict(out=X + 4), -1),
    ("overlaps", dict(out=X, out_dtype=1), -1), ("overlaps", dict(out=X, out_batch_stride=9000), -1),
    ("aligned", dict(x=X + 2), -3), ("aligned", dict(out=OUT + 1, out_dtype=1), -3), ("256", dict(ws=WS + 128), -3)])
def test_orthogonalize_refuses(what, kw, code):
    assert _orth(**kw) == code and what in ma.adam_last_error()


@pytest.mark.parametrize("steps,coefficients,eps", [(0, None, 1e-7), (17, None, 1e-7), (5, None, 0.0), (5, None, -1.0),
                                                    (5, None, float("inf")), (5, None, float("nan")),
                                                    (2, (1.0, 65.0, 0.0), 1e-7), (2, (1.0, float("nan"), 0.0), 1e-7)])
def test_orthogonalize_refuses_bad_iterations(steps, coefficients, eps):
    assert _orth(it=M._iteration(steps, coefficients, eps)) == -1


def test_empty_batches_need_no_memory():
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0, x_row_stride=0, out_row_stride=0)):
        assert _orth(x=0, out=0, ws=0, ws_bytes=0, **kw) == 0


def test_iterations_of_the_binding():
    it = M._iteration(2, [(1.5, -0.5, 0.0), (2.0, -1.5, 0.5)], 1e-3)
    assert it.steps == 2 and list(it.coefficients[:6]) == [1.5, -0.5, 0.0, 2.0, -1.5, 0.5]
    assert list(M._iteration(2, (3, -4, 2), 1e-3).coefficients[:6]) == [3, -4, 2, 3, -4, 2]
    assert not M._iteration(5, None, 1e-7).coefficients
    for bad in ([1.0, 2.0], [(1.0, 2.0, 3.0)], [(1.0, 2.0)] * 5, [(1.0, 2.0, 3.0)] * 6):
        with pytest.raises(ValueError):
            M._iteration(5, bad, 1e-7)


# ---------------------------------------------------------------- checkpoint stream
def _hash(b):
    h = (0x9E3779B97F4A7C15 ^ len(b)) & 0xFFFFFFFFFFFFFFFF
    for i in range(0, len(b) - 7, 8):
        h = ((h ^ int.from_bytes(b[i:i + 8], "little")) * 0x100000001B3) & 0xFFFFFFFFFFFFFFFF
        h ^= h >> 29
    return h ^ (h >> 32)


def _stream(shapes, storage=2, version=1, draw=None, records=None, options=0, block=2048):
    pad = [(r * c + 15) // 16 * 16 for r, c in shapes]
    draw = [sum(pad[:k]) for k in range(len(shapes))] if draw is None else draw
    blocks = sum(-(-r * c // 2048) for r, c in shapes)
    out = bytearray(b"MEAMMUON")
    out += struct.pack("<IIiiiIiI", version, 40 + 24 * len(shapes), storage, 0, block, options, len(shapes), 0)
    for v in ([r for r, _ in shapes], [c for _, c in shapes], draw):
        out += struct.pack(f"<{len(v)}q", *v)
    if records is None:
        records = {2: [(0, sum(pad)), (2, 4 * blocks)], 1: [(4, 2 * sum(pad))], 3: [(6, 4 * sum(pad))]}[storage]
    for bid, nb in records:
        out += struct.pack("<IIQ", bid, 0, nb) + bytes((nb + 7) // 8 * 8)
    out += struct.pack("<II", 0xFFFFFFFF, len(records))
    return bytes(out) + struct.pack("<Q", _hash(bytes(out)))


def _load(buf):
    h = ctypes.c_void_p()
    arr = (ctypes.c_uint8 * max(1, len(buf))).from_buffer_copy(buf or b"\0")
    rc = M.library().muon_state_load(ctypes.byref(h), ctypes.cast(arr, ctypes.c_void_p), len(buf), None)
    if rc == 0:
        M.library().muon_state_destroy(h)
    return rc


SHAPES = [(50, 100), (1, 17)]


def _rehash(b):
    return bytes(b[:-8]) + struct.pack("<Q", _hash(bytes(b[:-8])))


def _patched(at, value):
    b = bytearray(_stream(SHAPES))
    b[at:at + len(value)] = value
    return _rehash(b)


@pytest.mark.parametrize("name,stream", [
    ("empty", b""), ("magic", b"X" + _stream(SHAPES)[1:]), ("version", _stream(SHAPES, version=2)),
    ("storage", _stream(SHAPES, storage=2).replace(struct.pack("<i", 2), struct.pack("<i", 9), 1)),
    ("options", _stream(SHAPES, options=1)), ("block", _stream(SHAPES, block=1024)),
    ("truncated", _stream(SHAPES)[:-24]), ("odd size", _stream(SHAPES) + b"\0"), ("longer", _rehash(_stream(SHAPES) + bytes(8))),
    ("checksum", _stream(SHAPES)[:-1] + b"\xff"), ("record size", _stream(SHAPES, records=[(0, 5024), (2, 12)])),
    ("record order", _stream(SHAPES, records=[(2, 16), (0, 5040)])), ("record missing", _stream(SHAPES, records=[(0, 5040)])),
    ("draw unaligned", _stream(SHAPES, draw=[0, 5008])[:-8] + bytes(8)), ("draw negative", _stream(SHAPES, draw=[-16, 5008])),
    ("draw too large", _stream(SHAPES, draw=[0, 2 ** 62 - 16])), ("rows", _patched(40, struct.pack("<q", -3))),
    ("rows large", _patched(40, struct.pack("<q", 2 ** 40))), ("tensors", _patched(32, struct.pack("<i", -1))),
    ("tensors many", _patched(32, struct.pack("<i", 2 ** 30))), ("record bytes", _patched(96, struct.pack("<Q", 2 ** 63)))])
def test_load_refuses_malformed_streams_before_any_device_call(name, stream):
    assert _load(stream) == -1, (name, ma.adam_last_error())


@pytest.mark.parametrize("storage", [1, 2, 3])
def test_load_of_a_valid_stream_gets_past_validation(storage):
    # without a GPU the first device call is what fails
    assert _load(_stream(SHAPES, storage=storage)) in (0, -4, -5)


# ---------------------------------------------------------------- binding checks
def _state(shapes, grad_dtype=0, storage=2):
    return M.MuonState(None, shapes, M.muon_layout(storage, grad_dtype, 2048, 0), device=0)


def test_step_refuses_bad_tensors_before_any_call():
    st = _state([(10, 10), (7, 1)])
    ok = [torch.zeros(10, 10), torch.zeros(7, 1)]
    for params, grads, what in (
            ([torch.zeros(10, 10)], ok, "expected 2"), ([torch.zeros(100), torch.zeros(7, 1)], ok, "shape"),
            (ok, [torch.zeros(5, 20), torch.zeros(7, 1)], "shape"), (ok, [torch.zeros(10, 10), torch.zeros(8, 1)], "numel"),
            ([torch.zeros(10, 10, dtype=torch.float64), torch.zeros(7, 1)], ok, "dtype"),
            (ok, [torch.zeros(10, 10, dtype=torch.bfloat16), torch.zeros(7, 1)], "dtype"),
            ([torch.zeros(10, 10).T, torch.zeros(7, 1)], [torch.zeros(10, 20)[:, ::2], torch.zeros(7, 1)], "contiguous"),
            (ok, ok, "device")):
        with pytest.raises(ValueError, match=what):
            ma.muon_step(st, params, grads, **HP)
    with pytest.raises(TypeError):
        ma.muon_step(st, [None, torch.zeros(7, 1)], ok, **HP)
    with pytest.raises(ValueError, match="device"):
        ma.muon_step(_state([(10, 10)], 1), [torch.zeros(10, 10)], [torch.zeros(10, 10, dtype=torch.bfloat16)], **HP)
    empty = _state([(0, 5)])
    with pytest.raises(ValueError, match="scale"):
        ma.muon_step(empty, [torch.zeros(0, 5)], [torch.zeros(0, 5)], scale="adam", stream=0, **HP)
    with pytest.raises(ma.AdamError):  # reaches the library, which refuses a NULL state
        ma.muon_step(empty, [torch.zeros(0, 5)], [torch.zeros(0, 5)], stream=0, **HP)


def test_orthogonalize_refuses_bad_tensors_before_any_call():
    x = torch.zeros(3, 8, 8)
    for bad, what in ((torch.zeros(8), "rows, cols"), (torch.zeros(8, 8, dtype=torch.float16), "dtype"),
                      (torch.zeros(8, 16)[:, ::2], "contiguous"), (x.transpose(1, 2), "contiguous"),
                      (torch.zeros(1, 8).expand(8, 8), "overlap"), (torch.zeros(4, 6, 8, 8)[:, ::2].transpose(0, 1), "stride"),
                      (torch.zeros(8, 8, requires_grad=True), "gradient"), (x, "device")):
        with pytest.raises(ValueError, match=what):
            ma.muon_orthogonalize(bad)
    with pytest.raises(ValueError, match="shape"):
        ma.muon_orthogonalize(x, out=torch.zeros(3, 8, 9))
    with pytest.raises(ValueError, match="coefficients"):
        ma.muon_orthogonalize(x, coefficients=(1.0, 2.0))
    with pytest.raises(TypeError):
        ma.muon_orthogonalize([[1.0]])


def test_batches_with_one_stride_are_taken():
    big = torch.zeros(4, 3, 10, 12)
    f = M._matrices_of
    of = lambda t: f("x", tuple(t.shape), t.stride(), t.dtype)  # noqa: E731
    assert of(big) == (12, 10, 12, 120, 12, 0)
    assert of(big[:, :, :7, :5]) == (12, 7, 5, 120, 12, 0)
    assert of(big[:, 1]) == (4, 10, 12, 360, 12, 0)
    assert of(big[1, 2]) == (1, 10, 12, 0, 12, 0)
    assert of(big[:, :1, 3:4, :6]) == (4, 1, 6, 360, 6, 0)
    assert of(torch.zeros(1, 4).expand(5, 1, 4).bfloat16())[0] == 5
