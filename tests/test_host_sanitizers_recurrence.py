"""The host code of the gated recurrence's and the checkpoints' entry points under
AddressSanitizer and UndefinedBehaviorSanitizer, as test_host_sanitizers.py has
the rest: recurrence_api.cpp and api.cpp built with g++ into a library that takes
the kernels from the built one, and tests/test_recurrence_abi.py run against it.
No GPU is involved: every call there fails validation or is empty."""

import os
import subprocess
import sys

import pytest
from test_host_sanitizers import PKG, ROOT, runtime

from selective_state_space_23_amd import _lib


def test_recurrence_checks_are_clean_under_asan_and_ubsan(tmp_path):
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libmamba_hip.so is not built: run `python -m selective_state_space_23_amd.build`")
    asan, ubsan = runtime("libasan.so"), runtime("libubsan.so")
    if asan is None or ubsan is None:
        pytest.skip("g++ with the ASan/UBSan runtimes is not available")
    lib = tmp_path / "libmamba_hip_sanitized.so"
    cmd = ["g++", "-O1", "-g", "-std=c++17", "-fPIC", "-shared", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
           "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-o", str(lib),
           os.path.join(PKG, "csrc", "recurrence_api.cpp"), os.path.join(PKG, "csrc", "api.cpp"),
           "-L", PKG, "-lmamba_hip", f"-Wl,-rpath,{PKG}"]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-3000:]
    env = dict(os.environ)
    env.update(LD_PRELOAD=f"{asan}:{ubsan}", MAMBA_HIP_LIB=str(lib),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                          os.path.join(ROOT, "tests", "test_recurrence_abi.py")],
                         env=env, capture_output=True, text=True, cwd=ROOT, timeout=600)
    assert run.returncode == 0, (run.stdout[-3000:], run.stderr[-3000:])
    assert "passed" in run.stdout and "failed" not in run.stdout, run.stdout[-2000:]
