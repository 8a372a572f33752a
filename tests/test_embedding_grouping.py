"""The grouping of tokens by row, which the gradient and the step of rows sum by: each row's
positions have to lie together, or parts of its sum are taken for the whole.  On the CPU, by
grouping_model.cpp behind the runtime's own plan and arguments; the kernel itself is
tested in test_gpu_embedding_grouping.py on the same tokens."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from grouping_tokens import KINDS, ROWS, tokens_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GRAD, TABLE = 1 << 45, 1 << 46  # no memory: the model reads tokens alone


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "cols", "tokens", "table_stride", "value_stride")] + \
               [(n, ctypes.c_int32) for n in ("table_dtype", "value_dtype", "token_dtype")] + [("scale", ctypes.c_float)]


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    out = str(tmp_path_factory.mktemp("grouping") / "libgrouping_model.so")
    csrc = os.path.join(ROOT, "memory_efficient_adam_amd", "csrc")
    here = os.path.join(ROOT, "tests")
    subprocess.run(["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__",
                    "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "adam_runtime.cpp"), os.path.join(csrc, "embedding_runtime.cpp"),
                    os.path.join(here, "sanitize", "launch_stub.cpp"), os.path.join(here, "grouping_model.cpp"),
                    "-L", os.path.join(rocm, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(rocm, 'lib')}",
                    "-o", out], check=True)
    lib = ctypes.CDLL(out)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.embedding_gradient.argtypes = [ctypes.POINTER(Shape), vp, vp, vp, i32, vp, i64, vp]
    lib.embedding_gradient_workspace_bytes.argtypes = [i64, i64, i64]
    lib.embedding_gradient_workspace_bytes.restype = i64
    for name in ("model_keys", "model_order"):
        getattr(lib, name).restype = ctypes.POINTER(ctypes.c_uint32)
    return lib


def _grouped(lib, tokens, rows):
    """(rows by position, positions) as the sums are given them."""
    n = len(tokens)
    need = lib.embedding_gradient_workspace_bytes(n, rows, 4)
    whole = np.empty(need + 256, np.uint8)
    at = -(-whole.ctypes.data // 256) * 256
    shape = Shape(rows, 4, n, 4, 4, 0, 0, 1 if tokens.dtype == np.int64 else 0, 1.0)
    assert lib.embedding_gradient(ctypes.byref(shape), GRAD, tokens.ctypes.data, TABLE, 1, at, need, None) == 0
    return (np.ctypeslib.as_array(lib.model_keys(), (n,)).copy(), np.ctypeslib.as_array(lib.model_order(), (n,)).copy())


@pytest.mark.parametrize("ids", [np.int32, np.int64])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", ROWS)
def test_each_row_is_one_run(model, rows, kind, ids):
    for n in (3000, 16384, 65536):
        tokens = tokens_of(kind, n, rows, seed=n).astype(ids)
        keys, order = _grouped(model, tokens, rows)
        live = int(((tokens >= 0) & (tokens < rows)).sum())
        named = np.unique(tokens[(tokens >= 0) & (tokens < rows)])
        starts = np.flatnonzero(np.concatenate([[True], keys[1:live] != keys[:live - 1]]))
        assert len(starts) == len(named), f"{n} tokens: {len(named)} rows in {len(starts)} runs"
        assert np.array_equal(keys[starts], named)  # in the rows' order
        assert (keys[live:] == 0xFFFFFFFF).all()
        assert np.array_equal(np.sort(order[:live]), np.flatnonzero((tokens >= 0) & (tokens < rows)))
        assert np.array_equal(tokens[order[:live]], keys[:live])
