"""The host-side argument handling of the token-model operators under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: the library is built with the sanitizers on its host code only
and linked into a driver (tests/sanitize/lm_driver.c) whose calls all end before the HIP runtime is asked
to do anything.  The driver exits non-zero on a failed check, and any report aborts it."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "selective_state_space_22_amd", "csrc")
INCLUDE = ["-I", os.path.join(ROOT, "include")]
HIPCC = "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/lib/llvm/bin/clang"


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    return r.returncode, r.stdout + r.stderr


def test_host_side_of_the_token_model_operators_under_sanitizers(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("ROCm compilers not found")
    from selective_state_space_22_amd import build as lib_build

    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
             "-Wno-unused-command-line-argument"] + INCLUDE

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        return obj, _run([HIPCC] + flags + ["-c", "-o", obj, os.path.join(CSRC, src)])

    with ThreadPoolExecutor(8) as ex:
        results = list(ex.map(compile_one, lib_build.SOURCES))
    for obj, (rc, log) in results:
        assert rc == 0, log
    lib = str(tmp_path / "libmamba_san.so")
    rc, log = _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", lib] + [o for o, _ in results])
    assert rc == 0, log
    exe = str(tmp_path / "lm_driver")
    rc, log = _run([CLANG, "-std=c11", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all"] + INCLUDE + ["-o", exe, os.path.join(ROOT, "tests", "sanitize",
                    "lm_driver.c"), lib, f"-Wl,-rpath,{tmp_path}", "-lstdc++", "-lm"])
    assert rc == 0, log
    rc, log = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    assert rc == 0 and "all checks passed" in log, log
    assert "runtime error" not in log and "AddressSanitizer" not in log, log
