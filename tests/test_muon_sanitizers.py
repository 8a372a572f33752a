"""The Muon host tests against a host-only build of the library with
AddressSanitizer and UndefinedBehaviorSanitizer (kernel launchers stubbed), and
a fuzz of the checkpoint loader on it (CPU, no GPU)."""
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
sys.path.insert(0, os.path.join(HERE, "sanitize"))
import build_sanitized as S  # noqa: E402

pytestmark = pytest.mark.skipif(shutil.which("gcc") is None or shutil.which("g++") is None,
                                reason="needs gcc/g++")


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("sanitized") / "libmuon_host_san.so")
    csrc = os.path.join(ROOT, "memory_efficient_adam_amd", "csrc")
    stubs = [os.path.join(HERE, "sanitize", f) for f in ("launch_stub.cpp", "muon_launch_stub.cpp")]
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", *S.SAN,
                    "-I", os.path.join(S.ROCM, "include"), "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "adam_runtime.cpp"), os.path.join(csrc, "muon_runtime.cpp"), *stubs,
                    "-L", os.path.join(S.ROCM, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(S.ROCM, 'lib')}",
                    "-o", out], check=True)
    return out


def _run(code, timeout=600):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=S.env_with_sanitizers(),
                       capture_output=True, text=True, timeout=timeout)
    assert r.returncode == 0, r.stdout[-4000:] + "\n" + r.stderr[-4000:]
    return r.stdout


def _preamble(library):
    return ("import sys; sys.path[:0] = [%r, %r]; import memory_efficient_adam_amd._binding as B; "
            "B._LIB_PATH = %r\n" % (ROOT, HERE, library))


def test_host_calls_under_sanitizers(library):
    out = _run(_preamble(library) + "import pytest; sys.exit(pytest.main(['-q', '-x', '-p', 'no:cacheprovider', "
                                    "'tests/test_muon_host.py']))")
    assert " passed" in out


def test_checkpoint_loader_fuzz_under_sanitizers(library):
    out = _run(_preamble(library) + """
import random
import test_muon_host as T
rng = random.Random(99)
bases = [T._stream([(50, 100), (1, 17)], storage=s) for s in (1, 2, 3)] + [T._stream([]), T._stream([(0, 3), (1, 1)])]
bad = 0
for _ in range(3000):
    b = bytearray(rng.choice(bases))
    for _ in range(rng.randint(1, 3)):
        kind = rng.randrange(3)
        if kind == 0 and b:
            b[rng.randrange(len(b))] ^= 1 << rng.randrange(8)
        elif kind == 1 and len(b) >= 16:
            w = rng.choice((4, 8))
            at = rng.randrange(0, len(b) - w + 1) // w * w
            v = rng.choice([0, 1, 15, 0x7FFFFFFF, 0x80000000, 2 ** 32, 2 ** 62, 2 ** 63, 2 ** 64 - 1])
            b[at:at + w] = (v & (2 ** (8 * w) - 1)).to_bytes(w, 'little')
        else:
            del b[rng.randrange(len(b) + 1):]
    s = bytes(b)
    if rng.random() < 0.7:
        s = s[:len(s) - len(s) % 8]
    if len(s) >= 8 and rng.random() < 0.7:
        s = T._rehash(s)
    if T._load(s) not in (0, -1, -4, -5):
        bad += 1
print(bad, 'unexpected results')
sys.exit(1 if bad else 0)
""")
    assert "0 unexpected results" in out
