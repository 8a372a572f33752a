"""The embedding calls where no GPU is needed: what the library exports, sizes of
workspaces, every refusal of the C calls (before any device call) and of the
binding, and the host code under sanitizers."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import memory_efficient_adam_amd as ma
from memory_efficient_adam_amd import _binding as B
from memory_efficient_adam_amd import _embedding as E

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, t=1)
# far apart, and no memory: calls that are not refused have to end at a missing device
TABLE, VALUES, TOKENS, WORK, M, V, W = (k << 44 for k in range(1, 8))
without_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="would launch on pointers that are no memory")


def _shape(**kw):
    s = dict(rows=100, cols=40, tokens=3000, table_stride=40, value_stride=40, table_dtype=0, value_dtype=0, token_dtype=1,
             scale=1.0)
    s.update(kw)
    if "cols" in kw:
        s["table_stride"], s["value_stride"] = kw.get("table_stride", s["cols"]), kw.get("value_stride", s["cols"])
    return E.embedding_shape(*[s[n] for n, _ in E.embedding_shape._fields_])


def _lookup(table=TABLE, ids=TOKENS, out=VALUES, **kw):
    return E.library().embedding_lookup(ctypes.byref(_shape(**kw)), table, ids, out, None)


def _gradient(grad=VALUES, ids=TOKENS, table=TABLE, accumulate=0, ws=WORK, ws_bytes=1 << 40, **kw):
    return E.library().embedding_gradient(ctypes.byref(_shape(**kw)), grad, ids, table, accumulate, ws, ws_bytes, None)


def _step(table=TABLE, grad=VALUES, ids=TOKENS, ws=WORK, ws_bytes=1 << 40, state=(M, V, W), hp=None, layout=None, **kw):
    buffers = (ctypes.c_void_p * 12)()
    for name, at in zip(("m_f32", "v_f32", "vmax_f32"), state or ()):
        buffers[B.BUFFERS[name]] = at
    hp = hp or B.adam_hparams(1e-3, 0.9, 0.999, 1e-8, 0.0, 100.0, 1, 1, 0, 42)
    layout = layout or B._layout("f32", "f32")
    return E.library().embedding_adam_step(ctypes.byref(_shape(**kw)), table, grad, ids,
                                           ctypes.cast(buffers, ctypes.c_void_p) if state else None, ctypes.byref(hp),
                                           ctypes.byref(layout), ws, ws_bytes, None)


CALLS = [_lookup, _gradient, _step]


def test_exports_and_struct():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "embedding_mi355x.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(embedding_[a-z_]+)\s*\(", src)))
    assert len(names) == 4
    lib = ctypes.CDLL(ma.library_path())
    for n in names:
        assert hasattr(lib, n) and hasattr(ma, n), n
    assert ctypes.sizeof(E.embedding_shape) == 56 and E.embedding_shape.scale.offset == 52


def test_workspace_bytes():
    w = ma.embedding_gradient_workspace_bytes
    assert w(0, 0, 5) == 0 and w(5, 5, 0) == 0
    assert w(1, 5, 7) == w(2048, 2 ** 31 - 1, 2 ** 31 - 1) == 0  # few tokens need none
    for tokens, rows, cols in ((2049, 1, 1), (8192, 1000, 7), (8193, 1000, 7), (16384, 50304, 2048), (5000, 2 ** 31 - 1, 3)):
        n = w(tokens, rows, cols)
        # keys and positions, twice for more rows than 2^18; a byte a row; two fp32 rows and three counters a window of 32 or 64
        windows = -(-tokens // (32 if tokens <= 8192 else 64))
        exact = 8 * tokens * (2 if rows > 2 ** 18 else 1) + rows + windows * (8 * (-(-cols // 4) * 4) + 12 * -(-cols // 256))
        assert n % 256 == 0 and exact <= n <= exact + 7 * 256
    assert w(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1) > 2 ** 50
    for bad in ((-1, 5, 5), (5, -1, 5), (5, 5, -1), (2 ** 31, 5, 5), (5, 2 ** 31, 5), (5, 5, 2 ** 31)):
        with pytest.raises(ma.AdamError) as e:
            w(*bad)
        assert e.value.code == -1


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=2 ** 31), dict(cols=-1), dict(cols=2 ** 31), dict(tokens=-1), dict(tokens=2 ** 31),
    dict(table_stride=39), dict(table_stride=2 ** 41), dict(value_stride=-1), dict(value_stride=2 ** 41),
    dict(table_dtype=2), dict(value_dtype=-1), dict(token_dtype=2), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(rows=2 ** 31 - 1, table_stride=2 ** 40), dict(tokens=2 ** 31 - 1, value_stride=2 ** 40),
])
def test_shapes_outside_their_domain_are_refused(call, bad):
    assert call(**bad) == -1, bad


@pytest.mark.parametrize("call", CALLS)
def test_a_null_shape_is_refused(call):
    lib = E.library()
    assert lib.embedding_lookup(None, TABLE, TOKENS, VALUES, None) == -1
    assert lib.embedding_gradient(None, VALUES, TOKENS, TABLE, 0, WORK, 1 << 40, None) == -1
    assert lib.embedding_adam_step(None, TABLE, VALUES, TOKENS, None, None, None, WORK, 1 << 40, None) == -1


def test_pointers_that_are_missing_or_unaligned():
    for kw in (dict(table=None), dict(ids=None), dict(out=None)):
        assert _lookup(**kw) == -1 and "NULL" in ma.adam_last_error(), kw
    for kw in (dict(table=None), dict(ids=None), dict(grad=None), dict(ws=None)):
        assert _gradient(**kw) == -1 and "NULL" in ma.adam_last_error(), kw
        assert _step(**kw) == -1 and "NULL" in ma.adam_last_error(), kw
    assert _lookup(table=TABLE + 2) == _lookup(out=VALUES + 2) == _lookup(ids=TOKENS + 4) == -3
    assert _gradient(table=TABLE + 2) == _gradient(grad=VALUES + 2) == _gradient(ids=TOKENS + 4) == -3
    assert _gradient(ws=WORK + 128) == _step(ws=WORK + 128) == _step(table=TABLE + 4) == -3
    assert _gradient(table=TABLE + 1, table_dtype=1) == _gradient(grad=VALUES + 1, value_dtype=1) == -3
    assert _step(state=(M + 4, V)) == _step(state=(M, V + 8)) == -3


def test_the_workspace_has_to_suffice():
    need = ma.embedding_gradient_workspace_bytes(3000, 100, 40)
    assert _gradient(ws_bytes=need - 1) == -1 and str(need) in ma.adam_last_error()
    assert _step(ws_bytes=need - 1) == -1 and str(need) in ma.adam_last_error()


@without_gpu
def test_few_tokens_need_no_workspace():
    assert _gradient(ws=None, ws_bytes=0, tokens=2048) == _step(ws=None, ws_bytes=0, tokens=2048) == -5
    assert _gradient(ws=TABLE, ws_bytes=0, tokens=2048) == -5  # not looked at


def test_what_is_written_meets_nothing_else():
    table, values, tokens = 100 * 40 * 4, 3000 * 40 * 4, 3000 * 8
    for out in (TABLE, TABLE + table - 4, TABLE - values + 4, TOKENS, TOKENS + tokens - 4, TOKENS - values + 4):
        assert _lookup(out=out) == -1 and "overlaps" in ma.adam_last_error(), hex(out)
    for out in (VALUES, VALUES + values - 4, VALUES - table + 4, TOKENS, TOKENS - table + 4):
        assert _gradient(table=out) == -1 and "overlaps" in ma.adam_last_error(), hex(out)
    for out in (VALUES, VALUES + values - 16, VALUES - table + 16, TOKENS, TOKENS - table + 16):
        assert _step(table=out) == -1 and "overlaps" in ma.adam_last_error(), hex(out)
    need = ma.embedding_gradient_workspace_bytes(3000, 100, 40)
    for ws in (TABLE, TABLE - need + 256, TABLE + (table - 4) // 256 * 256, VALUES, TOKENS):
        assert _gradient(ws=ws) == -1 and "workspace" in ma.adam_last_error(), hex(ws)
        assert _step(ws=ws) == -1 and "workspace" in ma.adam_last_error(), hex(ws)
    for m in (TABLE, VALUES, TOKENS, WORK, V, V + table - 16, V - table + 16):
        assert _step(state=(m, V)) == -1 and "overlap" in ma.adam_last_error(), hex(m)
    ams = B._layout("f32", "f32", options=1)
    for w in (TABLE, VALUES, TOKENS, WORK, V, M + table - 16, None):
        assert _step(state=(M, V, w), layout=ams) == -1, w


def test_arguments_of_the_step():
    assert _step(state=None) == -1 and "state" in ma.adam_last_error()
    assert _step(state=(None, V)) == -1 and _step(state=(M, None)) == -1
    assert _step(layout=B._layout("q8", "f32")) == -2 and _step(layout=B._layout("bf16", "f32")) == -2
    assert _step(layout=B._layout("f32", "bf16")) == -2 and _step(value_dtype=1) == -2
    assert _step(layout=B._layout("f32", "f32", 1024)) == -1 and _step(layout=B._layout("f32", "f32", options=2)) == -1
    assert _step(table_dtype=1) == -1 and "fp32" in ma.adam_last_error()
    assert _step(table_stride=41) == -1 and "contiguous" in ma.adam_last_error()
    assert _step(rows=2 ** 16, cols=2 ** 16) == -1 and "2^32" in ma.adam_last_error()
    assert _step(rows=2 ** 31 - 1, cols=3) == -1 and "2^32" in ma.adam_last_error()
    for change in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0),
                   dict(weight_decay=-1.0), dict(t=0), dict(flags=2), dict(flags=4), dict(flags=8), dict(flags=16),
                   dict(reserved=1)):
        hp = B.adam_hparams(1e-3, 0.9, 0.999, 1e-8, 0.0, 100.0, 1, 1, 0, 42)
        for k, v in change.items():
            setattr(hp, k, v)
        assert _step(hp=hp) == -1, change


@without_gpu
def test_calls_that_are_not_refused_reach_the_device():
    table, values = 100 * 40 * 4, 3000 * 40 * 4
    assert _lookup() == _gradient() == _step() == -5
    assert _lookup(out=TABLE + table) == _lookup(out=TABLE - values) == -5
    assert _gradient(value_stride=0) == _gradient(value_stride=1000, table_stride=77) == -5
    assert _step(rows=2 ** 16, cols=2 ** 16 - 1) == _step(rows=2 ** 31 - 1, cols=2) == -5


def test_nothing_to_do_needs_no_device():
    assert _lookup(ids=None, table=None, out=None, cols=0) == 0
    s = _shape(tokens=0)
    lib = E.library()
    assert lib.embedding_lookup(ctypes.byref(s), None, None, None, None) == 0
    assert lib.embedding_gradient(ctypes.byref(s), None, None, TABLE, 1, None, 0, None) == 0
    assert _gradient(rows=0) == _gradient(cols=0) == _step(rows=0) == _step(cols=0) == 0


# ---------------------------------------------------------------- binding
def _raises(error, match, call, *args, **kw):
    with pytest.raises(error, match=match):
        call(*args, **kw)


def test_binding_refuses_host_tensors_and_others():
    table, tokens, grad = torch.zeros(5, 4), torch.zeros(3, dtype=torch.int64), torch.zeros(3, 4)
    buffers = {"m_f32": torch.zeros(32), "v_f32": torch.zeros(32)}
    if torch.cuda.device_count() > 0:
        pytest.skip("the checks of devices come with the GPU tests")
    B_current, B._current_device = B._current_device, lambda: 0
    try:
        _raises(ValueError, "device tensor", ma.embedding_lookup, table, tokens)
        _raises(ValueError, "device tensor", ma.embedding_gradient, grad, tokens, 5)
        _raises(ValueError, "device tensor", ma.embedding_adam_step, table, grad, tokens, buffers, **HP)
        _raises(TypeError, "torch tensor", ma.embedding_lookup, [[1.0]], tokens)
    finally:
        B._current_device = B_current


def test_a_captured_backward_pass_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    _raises(ValueError, "cannot be captured", E._function().backward, None, torch.zeros(3, 4))


def test_binding_checks_of_layouts():
    # the shape rules need no device
    assert E._row_stride("x", (3, 4), (4, 1)) == 4 and E._row_stride("x", (3, 4), (9, 1)) == 9
    assert E._row_stride("x", (3, 4), (0, 1)) == 0 and E._row_stride("x", (1, 4), (77, 1)) == 4
    assert E._row_stride("x", (2, 3, 4), (12, 4, 1)) == 4 and E._row_stride("x", (2, 3, 1), (15, 5, 3)) == 5
    assert E._row_stride("x", (2, 1, 4), (8, 3, 1)) == 8 and E._row_stride("x", (4,), (1,)) == 4
    assert E._row_stride("x", (2, 0, 4), (1, 1, 7)) == 4
    for shape, stride in (((3, 4), (1, 3)), ((2, 3, 4), (13, 4, 1)), ((3, 4), (4, 2))):
        _raises(ValueError, "rows must", E._row_stride, "x", shape, stride)
    _raises(ValueError, "dtype", E._dtype, "x", torch.float16)
    _raises(ValueError, "dtype", E._dtype, "tokens", torch.int16, E._TOKEN_DTYPES)


# ---------------------------------------------------------------- sanitizers
def test_host_code_under_sanitizers(tmp_path):
    import shutil
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    sys.path.insert(0, os.path.join(ROOT, "tests", "sanitize"))
    import build_sanitized as S
    out = str(tmp_path / "libembedding_host_san.so")
    csrc = os.path.join(ROOT, "memory_efficient_adam_amd", "csrc")
    here = os.path.join(ROOT, "tests", "sanitize")
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", *S.SAN,
                    "-I", os.path.join(S.ROCM, "include"), "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "adam_runtime.cpp"), os.path.join(csrc, "embedding_runtime.cpp"),
                    os.path.join(here, "launch_stub.cpp"), os.path.join(here, "embedding_launch_stub.cpp"),
                    "-L", os.path.join(S.ROCM, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(S.ROCM, 'lib')}",
                    "-o", out], check=True)
    code = f'''
import sys
sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, "tests")!r}]
from memory_efficient_adam_amd import _binding as B
B._LIB_PATH = {out!r}
import inspect, test_embedding_host as T
for name, f in sorted(vars(T).items()):
    if name in ("test_workspace_bytes", "test_pointers_that_are_missing_or_unaligned", "test_the_workspace_has_to_suffice",
                "test_what_is_written_meets_nothing_else", "test_arguments_of_the_step",
                "test_nothing_to_do_needs_no_device", "test_calls_that_are_not_refused_reach_the_device"):
        f(); print(name)
for mark in T.test_shapes_outside_their_domain_are_refused.pytestmark:
    if mark.args[0] == "bad":
        for bad in mark.args[1]:
            for call in T.CALLS:
                T.test_shapes_outside_their_domain_are_refused(call, bad)
print("done")
'''
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=S.env_with_sanitizers(), capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and "done" in r.stdout, (r.stdout[-3000:], r.stderr[-3000:])
