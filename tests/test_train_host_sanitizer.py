"""The host side of the training entry points (csrc/train_api.hip) under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: compiled as plain C++ with g++ against host-only
stand-ins of the kernel launchers (tests/host_sanitize/train_checks.cpp, which check that
nothing out of a kernel's range gets past the checks) and driven through a sweep of extreme
shapes and missing pointers."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_mixture_experts_sum_amd", "csrc")
ROCM_INCLUDE = "/opt/rocm/include"


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INCLUDE),
                    reason="needs g++ and the ROCm headers")
def test_training_host_code_under_asan_and_ubsan(tmp_path):
    exe = tmp_path / "train_checks"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-x", "c++", os.path.join(CSRC, "train_api.hip"),
           "-x", "c++", os.path.join(ROOT, "tests", "host_sanitize", "train_checks.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 and "asan" in (r.stdout + r.stderr).lower():
        pytest.skip("the sanitizer runtime is not installed: " + r.stderr[-300:])
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "passed: 0 failure(s)" in r.stdout
    assert "runtime error" not in out and "AddressSanitizer" not in out
