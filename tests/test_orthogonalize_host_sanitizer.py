"""The host side of the orthogonalisation (csrc/orthogonalize.hip: workspace layout, plans, launch sequence) under
AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: only the host part is compiled, with its
variables filled with a pattern, against stand-ins of the HIP runtime that look at every launch's buffers, their extents and grids
(tests/host_sanitize/orthogonalize_checks.cpp), for every path, type, number of steps and some 500 pairs of sides."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_mixture_experts_sum_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang++"


@pytest.mark.skipif(not os.path.exists(HIPCC) or not os.path.exists(CLANG), reason="needs hipcc")
def test_orthogonalize_host_code_under_asan_and_ubsan(tmp_path):
    obj, exe = tmp_path / "checks.o", tmp_path / "checks"

    def run(*cmd):
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
        if r.returncode != 0 and "libclang_rt" in r.stdout + r.stderr:
            pytest.skip("the sanitizer runtime is not installed: " + r.stderr[-300:])
        assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
        return r.stdout + r.stderr
    run(HIPCC, "-x", "hip", "--offload-host-only", "-O1", "-g", "-std=c++17", "-ftrivial-auto-var-init=pattern",
        "-Xarch_host", "-fsanitize=address,undefined", "-Xarch_host", "-fno-sanitize-recover=undefined",
        "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", os.path.join(ROOT, "tests", "host_sanitize", "orthogonalize_checks.cpp"),
        "-o", str(obj))
    # (the one symbol that stays open is the device code's, of which there is none)
    run(CLANG, "-fsanitize=address,undefined", "-no-pie", "-Wl,--unresolved-symbols=ignore-in-object-files", str(obj), "-o", str(exe))
    out = run(str(exe))
    assert "passed: 0 failure(s)" in out
    assert "runtime error" not in out and "AddressSanitizer" not in out
