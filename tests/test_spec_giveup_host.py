"""What the merge of the tree attention makes of a range whose bounded wait ran
out, on the host (shared host/device code of csrc/kvq_tree.cuh): flags that
such a range left unwritten never send it to drafted tokens that the call does
not have."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_abandoned_ranges(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "spec_giveup_check")
    subprocess.check_call([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-o", exe,
                           os.path.join(HERE, "spec_giveup_check.cu")])
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and "bad 0" in out.stdout, out.stdout[-2000:]
