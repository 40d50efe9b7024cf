"""Long caches: byte offsets past 32 bits in every operator over the cache, and
an eviction that selects among more groups than a CTA holds in registers."""
import numpy as np
import pytest
import torch

from _spec_testutil import config

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


@pytest.mark.parametrize("form,tokens", [("kv8", 20_000_036), ("fp16", 10_000_003)])
def test_offsets_past_32_bits(B, form, tokens):
    """A cache of zeros (logits of 0) but for its last 300 tokens, of which each
    query names one with a logit past 40: the second stream's codes lie past
    4 GB, and its result and record must come from there.  The zeros weigh
    less than 2e7 e^-40; the value read has its rounding (8 bits) and the
    output's."""
    free, _ = torch.cuda.mem_get_info()
    cfg = config(form, 1, 4, 2, tokens, softmax_scale=1.0)
    if free < 3 * B.kvq_layout_query(B.make_config(cfg)).layer_bytes // 2:
        pytest.skip("not enough device memory")
    g = torch.Generator(device="cuda").manual_seed(5)
    layer = B.Layer(cfg)
    k = torch.sign(torch.randn(1, 2, 300, 128, device="cuda", generator=g)).half()  # |k|^2 = 128; others within 60 of 0
    v = torch.randn(1, 2, 300, 128, device="cuda", generator=g).half()
    layer.append(tokens - 300, k, v)
    for n, named in ((2, (0, 150)), (40, (7, 299))):
        q = torch.zeros(1, 4, n, 128, device="cuda", dtype=torch.float16)
        for head in range(4):
            for i in range(n):
                q[0, head, i] = k[0, head // 2, named[i & 1]]
        out, lse, mass = torch.zeros_like(q), torch.zeros(1, 4, n, device="cuda"), B.new_mass(cfg)
        layer.tree_attn([tokens], q, None, None, None, out, lse, B.new_tree_workspace(cfg, n))
        layer.attn_mass([tokens], q, lse, mass)
        torch.cuda.synchronize()
        for head in range(4):
            for i in range(n):
                want = v[0, head // 2, named[i & 1]].float()
                # a step of 8-bit codes over a group's range of at most 9, half of it, and the output's rounding
                assert (out[0, head, i].float() - want).abs().max() <= 9 / 255 / 2 + 9 * 2.0 ** -9, (n, head, i)
        for s in range(2):
            for j in (0, 1):
                got = mass[0, s, tokens - 300 + named[j]].item()
                assert abs(got - n) <= 1e-3 * n, (n, s, j, got)  # two heads, half of the rows each
        del mass


def test_offsets_of_an_eviction(B):
    """The named tokens survive the departure of a thousand groups of zeros."""
    tokens = 20_000_036
    cfg = config("kv8", 1, 4, 2, tokens, softmax_scale=1.0)
    g = torch.Generator(device="cuda").manual_seed(6)
    layer = B.Layer(cfg)
    k = torch.sign(torch.randn(1, 2, 300, 128, device="cuda", generator=g)).half()
    v = torch.randn(1, 2, 300, 128, device="cuda", generator=g).half()
    layer.append(tokens - 300, k, v)
    q = torch.stack([k[0, h // 2, 100] for h in range(4)])[None, :, None].contiguous()
    ws, out, lse = B.new_tree_workspace(cfg, 1), torch.zeros_like(q), torch.zeros(1, 4, 1, device="cuda")
    layer.tree_attn([tokens], q, None, None, None, out, lse, ws)
    mass = torch.ones(1, 2, tokens, device="cuda")
    mass[0, :, tokens - 300:] = 2.0
    after = layer.evict([tokens], [1000], mass, mass, None, B.new_evict_workspace(cfg))
    assert after == [tokens - 32000]
    o2 = torch.zeros_like(q)
    layer.tree_attn(after, q, None, None, None, o2, lse, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, o2)  # the same token, its neighbours weigh e^-60
    assert mass[0, :, tokens - 32000:].abs().max().item() == 0
    assert (mass[0, :, :tokens - 32000] >= 1).all()
    assert [int((mass[0, s] == 2).sum()) for s in range(2)] == [300, 300]


@pytest.mark.parametrize("share", [0.001, 0.4, 0.98])
def test_many_groups(B, share):
    """5,900 groups a stream, sums of few values (ties), against the formula."""
    rng = np.random.default_rng(3)
    T = 32 * 5900 + 36 + 11
    cfg = config("kv2", 1, 2, 2, T)
    layer = B.Layer(cfg)
    groups = (T - 36) // 32
    mass = np.zeros((1, 2, T), np.float32)
    mass[0, :, 4:4 + 32 * groups] = rng.integers(0, 40, (2, 32 * groups)) * 0.25  # sums are exact
    mass[0, 1, 4:4 + 32 * groups] *= -1
    mass[0, :, 4 + 32 * groups:] = 5.0
    E = int(share * groups)
    source = torch.full((1, 2, groups), -1, dtype=torch.int32, device="cuda")
    record = torch.from_numpy(mass).cuda()
    layer.evict([T], [E], record, record, source, B.new_evict_workspace(cfg))
    torch.cuda.synchronize()
    left = groups - E
    for s in range(2):
        total = mass[0, s, 4:4 + 32 * groups].astype(np.float64).reshape(groups, 32)
        gone = np.zeros(groups, bool)
        gone[np.argsort(total.sum(1), kind="stable")[:E]] = True
        want = np.arange(left)
        want[gone[:left]] = left + np.flatnonzero(~gone[left:])
        assert (source[0, s, :left].cpu().numpy() == want).all()
        assert (source[0, s, left:] == -1).all()
        got = record[0, s].cpu().numpy()
        assert (got[4:4 + 32 * left].reshape(left, 32) == total[want]).all()
        assert (got[4 + 32 * left:T - 32 * E] == 5.0).all() and (got[T - 32 * E:] == 0).all()
