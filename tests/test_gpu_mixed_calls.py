"""Calls over a layer whose heads differ in bits that go wrong half way."""
import numpy as np
import pytest
import torch

from _spec_testutil import config, random_kv

pytestmark = pytest.mark.gpu
PAIRS = [(4, 4), (2, 2), (8, 8)]


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


def test_a_part_that_raises_leaves_the_others_joined(B):
    """What earlier parts launched on side streams comes before later work on
    the caller's stream, also when a part raises."""
    from bit_kv_cache_07_gb300.mixed import MixedLayer
    mixed = MixedLayer(config("kv4", 1, 3, 3, 300), PAIRS)
    x = torch.zeros(1 << 28, device="cuda")  # 1 GB: a pass takes a third of a millisecond
    parts = []

    def call(layer, ws, stream):
        parts.append(layer)
        if len(parts) == 3:
            raise ValueError("refused")
        if len(parts) == 2:
            with torch.cuda.stream(stream):
                for _ in range(50):
                    x.add_(1.0)

    torch.cuda.synchronize()
    with pytest.raises(ValueError):
        mixed._side_by_side(call, None)
    seen = x[-1:].clone()
    torch.cuda.synchronize()
    assert seen.item() == 50.0
