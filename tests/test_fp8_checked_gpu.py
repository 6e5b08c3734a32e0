"""The suites of the 8-bit products, quantisers, routing and combining run again on the checked
build with debug-sync on (GPU): every ordinary store of a product's C lies inside it and no
bounded wait gives up.  (Tests that capture a graph are left out: debug-sync waits for each call,
which a capture does not allow.)"""
import os
import subprocess
import sys

import pytest
import torch

import dense_gemm_05_gb300 as g

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_suites_pass_on_the_checked_build():
    if g.checked_requested():
        pytest.skip("this is the checked child process")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.build(checked=True)
    env = dict(os.environ, DG_GEMM_CHECKED="1", GEMM_DEBUG_SYNC="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-rs", "-m", "gpu", "-p", "no:cacheprovider",
           "-k", "not graph and not example", "tests/test_checked_gpu.py::test_the_checked_library_is_the_one_loaded",
           "tests/test_fp8_gpu.py", "tests/test_experts_gpu.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    tail = (r.stdout[-4000:] + "\n" + r.stderr[-2000:]).strip()
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "runs inside the checked child" not in r.stdout, tail
