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


def setup(B, seed=80):
    """A filled layer of three parts, its records and the state that a refused
    call must leave."""
    from bit_kv_cache_07_gb300.mixed import MixedLayer
    rng = np.random.default_rng(seed)
    mixed = MixedLayer(config("kv4", 2, 6, 3, 500), PAIRS)
    k, v = (torch.from_numpy(x).cuda() for x in random_kv(rng, (2, 3, 500, 128), big=False))
    mixed.append_ragged([0, 0], [500, 300], k, v)
    mass = mixed.new_mass()
    for m in mass:
        m.copy_(torch.from_numpy(rng.random(m.shape).astype(np.float32)))
    torch.cuda.synchronize()
    state = [x.clone() for x in [layer.buf for _, _, layer in mixed.parts] + mass]
    return mixed, mass, state


def unchanged(mixed, mass, state):
    torch.cuda.synchronize()
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
               for a, b in zip([layer.buf for _, _, layer in mixed.parts] + mass, state))


def test_an_eviction_refused_for_one_part_changes_none(B):
    mixed, mass, state = setup(B)
    ws, src = mixed.new_evict_workspace(), [torch.zeros(2, 1, 14, dtype=torch.int32, device="cuda") for _ in range(3)]
    for i in (1, 2):  # the part that is refused, after others that are not
        def put(values, x):
            return values[:i] + [x] + values[i + 1:]
        overlap = torch.zeros(2 * 500 + 32, device="cuda")
        for bad in (dict(mass=put(mass, mass[i].double())), dict(mass=put(mass, mass[i][:, :, :400].contiguous())),
                    dict(out=put(mass, mass[i].cpu())), dict(ws=put(ws, ws[i][:64])), dict(ws=put(ws, None)), dict(ws=put(ws, ws[i][8:])),
                    dict(src=put(src, src[i].long())), dict(src=put(src, src[i][:, :, :9].contiguous())),
                    dict(mass=put(mass, overlap[:1000].view(2, 1, 500)), out=put(mass, overlap[32:].view(2, 1, 500)))):
            a = dict(dict(mass=mass, out=mass, ws=ws, src=src), **bad)
            with pytest.raises((ValueError, TypeError, B.KvqError)):
                mixed.evict([500, 300], [2, 1], a["mass"], a["out"], a["src"], a["ws"])
            assert unchanged(mixed, mass, state), (i, list(bad))
    for tokens, drop in (([500, 301, 0], [1, 1, 0]), ([500, 501], [1, 1]), ([500, 300], [1, 9]), (iter([500, 300]), [1, 1])):
        with pytest.raises((ValueError, B.KvqError)):  # refused for every part
            mixed.evict(tokens, drop, mass, mass, src, ws)
        assert unchanged(mixed, mass, state)
    assert mixed.evict([500, 300], [2, 1], mass, mass, src, ws) == [436, 268]
    assert not unchanged(mixed, mass, state)


def test_a_record_refused_for_one_part_changes_none(B):
    mixed, mass, state = setup(B, 81)
    q, lse = torch.zeros(2, 6, 3, 128, dtype=torch.float16, device="cuda"), torch.full((2, 6, 3), 6.0, device="cuda")
    for i in (1, 2):
        for x in (mass[i].double(), mass[i][:, :, :400].contiguous(), mass[i].cpu(), None):
            with pytest.raises((ValueError, TypeError)):
                mixed.attn_mass([500, 300], q, lse, mass[:i] + [x] + mass[i + 1:])
            assert unchanged(mixed, mass, state), i
    mixed.attn_mass([500, 300], q, lse, mass)
    assert not unchanged(mixed, mass, state)


def test_parts_that_share_a_tensor_are_refused(B):
    """The parts run side by side: one scratch, record or source for two of
    them is a race."""
    mixed, mass, state = setup(B, 82)
    ws, src = mixed.new_evict_workspace(), [torch.zeros(2, 1, 14, dtype=torch.int32, device="cuda") for _ in range(3)]
    out = mixed.new_mass()
    big = torch.empty(ws[0].numel() + 64, dtype=torch.uint8, device="cuda")
    for bad in (dict(mass=[mass[0], mass[1], mass[0]], out=[mass[0], mass[1], mass[0]]), dict(out=[out[0], out[0], out[2]]),
                dict(src=[src[0], src[1], src[1]]), dict(ws=[ws[0], ws[0], ws[2]]), dict(ws=[big[:-64], ws[1], big[64:]]),
                dict(mass=[out[1], mass[1], mass[2]], out=out)):
        a = dict(dict(mass=mass, out=out, ws=ws, src=src), **bad)
        with pytest.raises(ValueError):
            mixed.evict([500, 300], [2, 1], a["mass"], a["out"], a["src"], a["ws"])
        assert unchanged(mixed, mass, state), list(bad)
    q, lse = torch.zeros(2, 6, 3, 128, dtype=torch.float16, device="cuda"), torch.full((2, 6, 3), 6.0, device="cuda")
    with pytest.raises(ValueError):
        mixed.attn_mass([500, 300], q, lse, [mass[0], mass[1], mass[0]])
    tree = mixed.new_tree_workspace(3)
    for shared in ([tree[0]] * 3, [tree[0], tree[1], tree[1][16:]]):
        with pytest.raises(ValueError):
            mixed.tree_attn([500, 300], q, None, None, None, q.clone(), lse, shared)
    assert unchanged(mixed, mass, state)
    # one record read by two parts is no race
    mixed.evict([500, 300], [2, 1], [mass[0], mass[1], mass[0]], out, src, ws)
    mixed.tree_attn([436, 268], q, None, None, None, q.clone(), lse, tree)
    torch.cuda.synchronize()


def test_one_part_takes_a_stream_handle(B):
    """A layer of equal heads is one part and takes the streams that its Layer takes."""
    from bit_kv_cache_07_gb300.mixed import MixedLayer
    rng = np.random.default_rng(83)
    cfg = config("kv4", 1, 4, 2, 300)
    k, v = (torch.from_numpy(x).cuda() for x in random_kv(rng, (1, 2, 300, 128), big=False))
    q, lse = torch.zeros(1, 4, 2, 128, dtype=torch.float16, device="cuda"), torch.full((1, 4, 2), 6.0, device="cuda")
    got = []
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        mixed = MixedLayer(cfg, [(4, 4)] * 2)
        mixed.append(0, k, v)
        mass, ws = mixed.new_mass(), mixed.new_evict_workspace()
        torch.cuda.synchronize()
        mixed.attn_mass([300], q, lse, mass, stream=stream)
        assert mixed.evict([300], [3], mass, mass, None, ws, stream=stream) == [204]
        torch.cuda.synchronize()
        got.append((mass[0], mixed.parts[0][2].buf))
    assert all(torch.equal(a, b) for other in got[1:] for a, b in zip(got[0], other))


def test_a_tree_refused_for_one_part_starts_none(B):
    mixed, mass, state = setup(B, 84)
    q, lse = torch.zeros(2, 6, 3, 128, dtype=torch.float16, device="cuda"), torch.full((2, 6, 3), 6.0, device="cuda")
    out, ws = torch.full_like(q, 7.0), mixed.new_tree_workspace(3)
    for i in (1, 2):
        for x in (ws[i][:4096], ws[i][8:], ws[i].cpu(), None):
            with pytest.raises((ValueError, TypeError, B.KvqError)):
                mixed.tree_attn([500, 300], q, None, None, None, out, lse, ws[:i] + [x] + ws[i + 1:])
            torch.cuda.synchronize()
            assert (out == 7.0).all() and (lse == 6.0).all()
    mixed.tree_attn([500, 300], q, None, None, None, out, lse, ws)
    torch.cuda.synchronize()
    assert (out != 7.0).any() and (lse != 6.0).all() and unchanged(mixed, mass, state)
