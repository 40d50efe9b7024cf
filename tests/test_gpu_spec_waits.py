"""The tile kernels' waits are bounded: one that nothing ends runs out, and the
context stays usable (spec_wait_check.cu).  What such a range leaves to the
merge is tested on the host (test_spec_giveup_host.py)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.gpu
def test_a_wait_runs_out(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "spec_wait_check")
    subprocess.check_call([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-o", exe,
                           os.path.join(HERE, "spec_wait_check.cu")])
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and "bad 0" in out.stdout, out.stdout[-2000:]
