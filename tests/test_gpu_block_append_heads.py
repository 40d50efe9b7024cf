"""kvq_block_append where a block's CTA takes several heads (calls of many rows per SM, see
append_split in csrc/kvq_block.cuh): against 64 bits and against calls of one head per CTA.
The split follows from the token slots, so that steps of few tokens run it, too."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_kv_cache_07_gb300 import blocks  # noqa: E402
from tests._block_testutil import BLOCK, D, EPS  # noqa: E402
from tests.test_gpu_block_append import Cache  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


def per_sm(n_tokens, hq, hkv):
    """CTAs of one head per SM; 3 and more heads of them make a CTA: by thirds up to 4 heads, by eighths beyond."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return n_tokens * (2 * hkv + hq) // (2 * BLOCK * sms)


def slots(rows, hq, hkv):
    """Token slots that give per_sm `rows`."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return -(-rows * 2 * BLOCK * sms // (2 * hkv + hq))


# heads of a CTA: 2 and 1, 4 and 3, 4 and 4 and 3, 3 of 5 (evenly 3 and 2), 8 and 7 by eighths
SPLITS = [(6, 3, 3), (12, 7, 7), (12, 11, 11), (9, 5, 5), (70, 30, 15)]
STEPS = [[40, 0, 3], [1, 70, 33], [31, 1, 64], [5, -1, 1], [1, 100, 1]]


@pytest.mark.parametrize("rows,hq,hkv", SPLITS)
@pytest.mark.parametrize("norm,theta,fused", [(True, 10000.0, True), (False, 0.0, False)])
def test_against_64_bits(rows, hq, hkv, norm, theta, fused):
    n = slots(rows, hq, hkv)
    assert per_sm(n, hq, hkv) == rows
    c = Cache(3, n, hq, hkv, 30, 9, seed=rows + hq, rope_theta=theta)
    x = np.zeros((n, hq + 2 * hkv, D), np.float16)  # rows behind the step's are not read
    for i, new in enumerate(STEPS):
        used = sum(max(0, v) for v in new)
        small = c.rng.standard_normal((used, hq + 2 * hkv, D)) * [1.0, 4.0, 0.25, 16.0, 1.0][i]
        small[:, hq:hq + hkv, :3] *= 8
        x[:] = np.nan
        x[:used] = small
        wq, wk = c.weights() if norm else (None, None)
        c.append(new, x, wq, wk, fused, queries=i != 2)
        c.check()


@pytest.mark.parametrize("rows,hq,hkv", SPLITS)
def test_the_bytes_of_one_head_per_cta(rows, hq, hkv):
    """The same steps with as many token slots as tokens: one head per CTA, the same bytes."""
    rng = np.random.default_rng(rows)
    caches = []
    many = slots(rows, hq, hkv)
    for n in (200, many):
        cfg = dict(batch=3, n_tokens=n, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, n_blocks=30, max_blocks=9, rope_theta=10000.0, norm_eps=EPS)
        caches.append((n, blocks.Tables(cfg), blocks.Layer(cfg)))
    assert per_sm(200, hq, hkv) < 6 <= per_sm(many, hq, hkv)
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal((2, D))).astype(np.float16)).cuda()
    for new in STEPS:
        used, outs = sum(max(0, v) for v in new), []
        x = torch.from_numpy(rng.standard_normal((used, hq + 2 * hkv, D)).astype(np.float16)).cuda()
        for n, t, layer in caches:
            g = torch.zeros((n, hq + 2 * hkv, D), dtype=torch.float16, device="cuda")
            g[:used] = x
            out = torch.full((n, hq, D), 7.0, dtype=torch.float16, device="cuda")
            t.plan(torch.tensor(new, dtype=torch.int32, device="cuda"))
            layer.append(t, g[:, hq:hq + hkv], g[:, hq + hkv:], g[:, :hq], out, w[0], w[1])
            assert (out[used:] == 7.0).all()
            outs.append(out[:used])
        assert torch.equal(*outs)
        assert torch.equal(caches[0][2].scales, caches[1][2].scales) and torch.equal(caches[0][2].codes, caches[1][2].codes)


@pytest.mark.parametrize("rows,hq,hkv", SPLITS[:3])
def test_not_finite_in_one_head(rows, hq, hkv):
    """A key that is not finite marks its head's block, not the CTA's other heads'."""
    n = slots(rows, hq, hkv)
    cfg = dict(batch=2, n_tokens=n, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, n_blocks=6, max_blocks=3)
    t, layer = blocks.Tables(cfg), blocks.Layer(cfg)
    t.plan(torch.tensor([40, 7], dtype=torch.int32, device="cuda"))
    k, v = torch.randn((n, hkv, D), device="cuda").half(), torch.randn((n, hkv, D), device="cuda").half()
    k[35, 1, 3], v[2, hkv - 1, 100] = float("inf"), float("nan")
    layer.append(t, k, v)
    marked = (layer.scales == 255).nonzero().tolist()
    a, b = t.block_table[0, :2].tolist()
    assert sorted(marked) == sorted([[b, 1, 0], [a, hkv - 1, 1]])
    assert int(((layer.codes & 127) == 127).sum()) == 0
