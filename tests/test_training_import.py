"""The binding of the training operators on a machine without a GPU."""
import os
import subprocess
import sys

import sparse_mixture_experts_sum_amd as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_with_a_torch_that_has_no_gpu_streams():
    # the host-only functions need no GPU, nor a torch built for one
    if not os.path.exists(M.LIB_PATH):
        from sparse_mixture_experts_sum_amd import build
        build.build()
    code = ("import torch; del torch._C._cuda_getCurrentRawStream; import sparse_mixture_experts_sum_amd as M; "
            "assert M.capacity(M.make_shape(8, 64, 64, 4, mode='tc_capacity')) > 0")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
