"""The block attention's waits are bounded: where one runs out, the kernel ends, the
rows that it was for become NaN and the others are right (block_wait_check.cu)."""
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("block") / "block_wait_check")
    subprocess.check_call([nvcc, "-O2", "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-o", exe,
                           os.path.join(HERE, "block_wait_check.cu")])

    def run(*args):
        out = subprocess.run([exe, *args], capture_output=True, text=True, timeout=120)
        assert out.returncode == 0 and "bad 0" in out.stdout, out.stdout[-2000:]
    return run


def test_every_wait_runs_out(check):
    check()


def test_one_wait_runs_out(check):
    """A chosen wait of one warp, or of one lane of it, at a range's begin and later."""
    check("later")
