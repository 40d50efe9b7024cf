"""Tree attention, the record and eviction of a layer whose heads differ in
bits, against uniform layers of each pair over the same tokens (whose own
results are compared with 64 bits elsewhere).  The grids differ, so sums are
cut elsewhere: each side is within (2^-11 + 2^-11) max |v| of the exact
attention of its stored values (values and output round once), and logits
within 2^-18 of sum |q k| scale, which is below 1 here."""
import numpy as np
import pytest
import torch

from _spec_testutil import config, random_kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


@pytest.mark.parametrize("pairs", [[(4, 4), (2, 8), (4, 4), (8, 2)], [(4, 2)] * 4])
@pytest.mark.parametrize("n", [3, 40])
def test_against_uniform_layers(B, pairs, n):
    from bit_kv_cache_07_gb300.mixed import MixedLayer
    rng = np.random.default_rng(11)
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    lengths, hkv, hq = [900, 333], 4, 8
    base = config("kv4", 2, hq, hkv, 1000)
    k, v = (t(x) for x in random_kv(rng, (2, hkv, 900, 128), big=False))
    q = t(rng.standard_normal((2, hq, n, 128)).astype(np.float16))
    kd, vd = (t(x) for x in random_kv(rng, (2, hkv, n, 128), big=False))
    words = B.tree_mask([[i - 1 for i in range(n)], [max(0, i - 2) if i else -1 for i in range(n)]]).cuda()
    drop, records = [5, 2], rng.integers(0, 50, (2, hkv, 1000)).astype(np.float32)

    mixed = MixedLayer(base, pairs)
    mixed.append_ragged([0, 0], lengths, k, v)
    out, lse, mass = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda"), mixed.new_mass()
    mixed.tree_attn(lengths, q, kd, vd, words, out, lse, mixed.new_tree_workspace(n))
    mixed.attn_mass(lengths, q, lse, mass)
    marks = [t(np.ascontiguousarray(records[:, heads])) for _, heads, _ in mixed.parts]
    assert mixed.evict(lengths, drop, marks, marks, None, mixed.new_evict_workspace()) == [900 - 160, 333 - 64]
    o2 = torch.zeros_like(out)
    mixed.tree_attn([740, 269], q, kd, vd, words, o2, None, mixed.new_tree_workspace(n))
    torch.cuda.synchronize()

    tol = 2 * 2.0 ** -10 * max(v.abs().max().item(), vd.abs().max().item())
    for part, (pair, heads, _) in enumerate(mixed.parts):
        cfg = dict(base, k_bits=pair[0], v_bits=pair[1])
        layer, ws = B.Layer(cfg), B.new_tree_workspace(cfg, n)
        layer.append_ragged([0, 0], lengths, k, v)
        w, wl, wm = torch.zeros_like(q), torch.zeros_like(lse), B.new_mass(cfg)
        layer.tree_attn(lengths, q, kd, vd, words, w, wl, ws)
        layer.attn_mass(lengths, q, wl, wm)
        mark = t(records)
        layer.evict(lengths, drop, mark, mark, None, B.new_evict_workspace(cfg))
        w2 = torch.zeros_like(q)
        layer.tree_attn([740, 269], q, kd, vd, words, w2, None, ws)
        torch.cuda.synchronize()
        rows = [h * 2 + j for h in heads for j in range(2)]
        assert (out[:, rows].float() - w[:, rows].float()).abs().max() <= tol
        assert (o2[:, rows].float() - w2[:, rows].float()).abs().max() <= tol
        assert (lse[:, rows] - wl[:, rows]).abs().max() <= 2.0 ** -17
        assert torch.allclose(mass[part], wm[:, heads], rtol=2.0 ** -15, atol=1e-7)
        assert torch.equal(marks[part], mark[:, heads])


def test_refused_lists(B):
    from bit_kv_cache_07_gb300.mixed import MixedLayer
    base = config("kv4", 1, 2, 2, 300)
    mixed = MixedLayer(base, [(4, 4), (2, 2)])
    q = torch.zeros(1, 2, 1, 128, dtype=torch.float16, device="cuda")
    lse = torch.zeros(1, 2, 1, device="cuda")
    for ws in (None, mixed.new_tree_workspace(1)[:1], mixed.new_tree_workspace(1)[0]):
        with pytest.raises(ValueError):
            mixed.tree_attn([10], q, None, None, None, q.clone(), lse, ws)
    with pytest.raises(ValueError):
        mixed.attn_mass([10], q, lse, B.new_mass(base))
    with pytest.raises(ValueError):
        mixed.evict([200], [1], mixed.new_mass(), mixed.new_mass(), [None], mixed.new_evict_workspace())
