"""kvq_block_plan_back without a GPU: what it refuses before any launch."""
import ctypes as C

import pytest

from bit_kv_cache_07_gb300 import binding, blocks


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


A = 1 << 20  # an address that is never read


def test_refusals():
    L = binding.lib()
    c = blocks.make_config(dict(batch=4, n_tokens=8, n_q_heads=8, n_kv_heads=2, head_dim=128, n_blocks=33, max_blocks=5))
    t = binding.kvq_block_tables(*[A for _ in binding.BLOCK_TABLES])
    ok = [C.byref(c), C.byref(t), A, A, A, A, None]
    for i, bad in ((0, None), (1, None), (2, None), (3, None), (4, None), (2, A + 2), (3, A + 1), (4, A + 2), (5, A + 2), (5, A + 1)):
        args = list(ok)
        args[i] = bad
        assert L.kvq_block_plan_back(*args) == -1, (i, bad)
    c.batch = 2000
    assert L.kvq_block_plan_back(*ok) == -2
