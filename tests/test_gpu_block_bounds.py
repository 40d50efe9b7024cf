"""kvq_block_attn within each row's own bounds (_block_bounds.py; test_block_bounds_host.py
plants mistakes that fall outside of them): the values' path, token for token, over whole,
cut and joined segments, windows, 8 to 64 rows, and the weights' two fp16 parts."""
import random

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests._block_bounds import check, naming, parts_of, two_level  # noqa: E402
from tests.test_gpu_block_attn import LENS, Pool  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


@pytest.mark.parametrize("lens,new", LENS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 1), (8, 2), (16, 1)])
def test_random_values(lens, new, hq, hkv):
    p = Pool(lens, new, hq, hkv, seed=sum(lens) + 3 * hq)
    check(p, *p.run())


@pytest.mark.parametrize("window,first", [(1, 0), (31, 3), (64, 33), (700, 5), (2500, 0)])
@pytest.mark.parametrize("lens,new", [LENS[4], LENS[7], ([1, 33, 3000, 700], [1, 1, 1, 1])])
def test_window(window, first, lens, new):
    p = Pool(lens, new, 8, 2, seed=window + first, window=window, n_first=first)
    check(p, *p.run())


@pytest.mark.parametrize("new", [1, 2, 4, 9, 17])  # 8, 8, 16, 64 rows; 64 and a second pass
@pytest.mark.parametrize("lens", [[300, 40], [3000, 33, 96], [12000], [9000, 1000, 5000, 31]])
def test_values_that_name_their_tokens(lens, new):
    """A value row left out, taken twice or exchanged with another shows at its channel."""
    p = Pool(lens, [min(new, n) for n in lens], 4, 1, seed=new)
    naming(p)
    rows = None if sum(p.new) < 12 else {0, 1, new // 2, new - 1, len(p.q) // 2, len(p.q) - 1}
    check(p, *p.run(), rows)


@pytest.mark.parametrize("lens,new,hq,hkv", [([64], [1], 4, 1), ([1000], [1], 4, 1), ([5000, 96, 700], [1, 1, 1], 8, 1), ([900], [2], 4, 1),
                                             ([20000], [1], 2, 1)])
def test_two_parts_of_a_weight(lens, new, hq, hkv):
    """Up to 8 rows of a KV head weights have 22 bits: those that round badly to 11, all in one direction."""
    p = Pool(lens, new, hq, hkv, seed=3)
    assert abs(two_level(p)) > 0.9 * 2.0**-11 and parts_of(p.cfg) == 2
    check(p, *p.run())


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    r = random.Random(seed + 100)
    B, hkv, g = r.choice([1, 2, 5, 17]), r.choice([1, 2, 3]), r.choice([1, 2, 4, 7, 12])
    top = r.choice([40, 300, 1500]) if B * hkv * g > 60 else r.choice([700, 6000])
    lens = [r.randint(1, r.choice([40, top])) for _ in range(B)]
    new = [min(n, r.choice([0, 1, 1, 1, 2, 5, r.randint(1, 20)])) for n in lens]
    cfg = dict(window=r.choice([1, 17, 64, 500]), n_first=r.choice([0, 4, 33])) if r.random() < 0.5 else {}
    p = Pool(lens, new, g * hkv, hkv, seed=seed, n_tokens=max(1, sum(new)) + r.choice([0, 0, 9]), pad_batch=r.choice([0, 3]), **cfg)
    if seed % 2:
        naming(p)
    rows = set(r.sample(range(len(p.q)), min(len(p.q), 24)))
    check(p, *p.run(), rows)


def test_wide_value_scales():
    """Value scales tens of octaves apart: each channel's own terms."""
    p = Pool([400, 100], [1, 3], 4, 2, seed=7)
    p.scales[:, :, 1] = np.random.default_rng(1).integers(100, 135, p.scales[:, :, 1].shape)
    check(p, *p.run())
