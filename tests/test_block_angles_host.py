"""The rotation's frequencies on the host against 60 digits: within 2^-54 of a turn for a
base of 1 or more, so that the angle at position p is off by less than p 2^-54 turns
(a power in doubles, off by an ulp, times 1 / 2 pi: 0.16 (2^-52 + 2^-53 + 2^-53) < 2^-53.6,
and the cut to 64 bits)."""
import os
import shutil
import subprocess
from decimal import Decimal, getcontext

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
BASES = ["1", "1.5", "100", "10000", "500000", "1000000", "1e10", "3.3e38"]


def test_frequencies(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "block_angle_check")
    subprocess.check_call([nvcc, "-O2", "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-o", exe,
                           os.path.join(HERE, "block_angle_check.cu")])
    lines = subprocess.run([exe, *BASES], capture_output=True, text=True, check=True).stdout.splitlines()
    getcontext().prec = 70
    for base, line in zip(BASES, lines, strict=True):
        b = Decimal(float(np.float32(base)))
        got = [int(x) for x in line.split()]
        assert len(got) == 64
        for i, f in enumerate(got):
            turns = (-(b.ln() * (2 * i)) / 128).exp() / (2 * PI) % 1
            off = abs(Decimal(f) / Decimal(2) ** 64 - turns)
            assert min(off, 1 - off) < Decimal(2) ** -54, (base, i, off)
