"""Scales that the append does not give (the caller's own): value scales far below its
least, and past its largest.  Bounds as in test_gpu_block_attn.py; what a scale below
2^-40 loses is below 448 * 2^-40 < 2^-31, a part of that bound's 2^-25."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests._block_testutil import attention, values  # noqa: E402
from tests.test_gpu_block_attn import Pool  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


@pytest.mark.parametrize("new", [1, 5, 20])  # 8, 32 and 64 rows
@pytest.mark.parametrize("some", [True, False])
def test_small_value_scales(some, new):
    """Their keys keep their weight in the sum, beside others and alone."""
    p = Pool([400, 100, 40], [new, new, new], 4, 2, seed=new)
    low = np.random.default_rng(2).integers(0, 87, p.scales[:, :, 1].shape)
    low[::3] = 0
    p.scales[:, :, 1] = np.where(np.random.default_rng(3).random(low.shape) < (0.5 if some else 1.0), low, p.scales[:, :, 1])
    p.check(*p.run())


def test_the_whole_range_of_the_append():
    """Value scales from 2^-40 to 2^20 side by side, those past 2^4 on small codes (out
    is fp16: 7 * 2^-9 * 2^20 < 65504)."""
    p = Pool([700, 90], [2, 1], 4, 2, seed=4)
    e = np.random.default_rng(5).integers(-40, 21, p.scales[:, :, 1].shape)
    p.scales[:, :, 1] = 127 + e
    p.codes[:, :, 1] = np.where((e > 4)[..., None, None], p.codes[:, :, 1] & 0x87, p.codes[:, :, 1])
    p.check(*p.run())


@pytest.mark.parametrize("byte", [168, 200, 254])
def test_large_value_scales_are_nan(byte):
    p = Pool([300, 300], [1, 1], 4, 2, seed=6)
    p.scales[p.table[0, 3], 1, 1] = byte
    p.codes[p.table[0, 3], 1, 1] = 0
    out, lse = p.run()
    p.check(out, lse, skip=(0,))
    assert np.isnan(out[0, 2:]).all() and np.isnan(lse[0, 2:]).all() and np.isfinite(out[0, :2]).all()
    p.scales[p.table[0, 3], 1, 1] = 167  # the largest that counts
    p.check(*p.run())


def test_least_key_scale():
    """Keys of scale 2^-127: logits of zero.  lse is (ref + log2 l) ln 2 with log2 l below
    32, whose ulp is 2^-19 at most."""
    p = Pool([100], [2], 4, 2, seed=7)
    p.scales[:, :, 0] = 0
    out, lse = p.run()
    kv = values(p.codes, p.scales)
    o, s = attention(p.q, kv, p.table[0], 100, 2, 4, 2)
    assert (np.abs(lse - s) <= 2.0**-19).all()
    assert (np.abs(out - o) <= 2.0**-10 * np.abs(kv[:, :, 1]).max()).all()
