"""kvq_attn_mass on the GPU against the weights in 64 bits.

Tolerance.  A weight's exponent carries the logit's error, E = 2^-20 scale
sum |q k| (22-bit keys, fp32 accumulation over 128 products), the fp32
rounding of the difference to lse (2^-24 of its size, below 2^-17 for the
sizes here) and the exponential's 2^-22; the sum of n weights rounds n times:
  |err| <= (e^E - 1 + 2^-16 + n 2^-24) sum + 2^-23 |decay mass|."""
import numpy as np
import pytest
import torch

from _spec_testutil import FORMS, cached, config, fill, random_kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


def check(B, cfg, lengths, n, seed, weights=False, decay=1.0, passes=1, more=0.0):
    rng = np.random.default_rng(seed)
    layer, stores = fill(B, cfg, lengths, rng)
    batch, hq, hkv, cap = cfg["batch"], cfg["n_q_heads"], cfg["n_kv_heads"], cfg["max_tokens"]
    g = hq // hkv
    q = rng.standard_normal((batch, hq, n, 128)).astype(np.float16)
    w = None
    if weights:
        w = np.where(rng.random((batch, n)) < 0.5, 0.0, rng.random((batch, n))).astype(np.float32)
        w[:, 0] = 0.0
        q[:, :, 0] = np.nan  # a row that does not count
    start = rng.random((batch, hkv, cap)).astype(np.float32)
    scale = np.float64(np.float32(cfg["softmax_scale"] or 1 / np.sqrt(128.0)))
    z, lse = {}, np.full((batch, hq, n), -np.inf, np.float32)
    for s, store in enumerate(stores):
        b, h = divmod(s, hkv)
        k = cached(cfg, store, lengths[b])[0]
        qs = q[b, h * g:(h + 1) * g].astype(np.float64)
        z[s] = scale * (qs @ k.T), scale * (np.abs(qs) @ np.abs(k).T)
        if lengths[b]:
            m = z[s][0].max(-1)
            lse[b, h * g:(h + 1) * g] = m + np.log(np.exp(z[s][0] - m[..., None]).sum(-1)) + more * rng.random((g, n))
    mass = torch.from_numpy(start.copy()).cuda()
    t = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    for _ in range(passes):
        layer.attn_mass(lengths, t(q), t(lse), mass, t(w), decay)
    torch.cuda.synchronize()
    got = mass.cpu().numpy()
    for s in range(batch * hkv):
        b, h = divmod(s, hkv)
        T = lengths[b]
        assert np.array_equal(got[b, h, T:], start[b, h, T:]), "entries past the tokens changed"
        if not T:
            continue
        p = np.exp(z[s][0] - lse[b, h * g:(h + 1) * g].astype(np.float64)[..., None])
        if w is not None:
            p[:, w[b] == 0] = 0.0
            p = p * w[b].astype(np.float64)[None, :, None]
        E = np.where(p > 0, z[s][1], 0.0).max() * 2.0 ** -20
        add = p.sum((0, 1))
        ref = start[b, h, :T].astype(np.float64)
        for _ in range(passes):
            ref = np.float64(np.float32(decay)) * ref + add
        bound = passes * ((np.expm1(E) + 2.0 ** -16 + g * n * 2.0 ** -24) * add + 2.0 ** -23 * np.abs(ref) + 2.0 ** -23 * start[b, h, :T])
        assert (np.abs(got[b, h, :T] - ref) <= bound).all(), (b, h, np.max(np.abs(got[b, h, :T] - ref) / bound))


LENGTHS = [0, 1, 35, 36, 67, 68, 300, 997]


@pytest.mark.parametrize("form", sorted(FORMS))
def test_forms(B, form):
    check(B, config(form, 8, 4, 2, 1024), LENGTHS, 1, 1)


@pytest.mark.parametrize("form", ["kv8", "kv2", "k4v2", "innerq4", "nuq", "kv4_rope", "fp16"])
@pytest.mark.parametrize("g,n", [(1, 1), (3, 5), (8, 1), (8, 8), (7, 37), (2, 129)])
def test_rows(B, form, g, n):
    check(B, config(form, 2, 2 * g, 2, 400, n_sink=0, n_recent=17), [333, 48], n, 2, weights=n > 1, decay=0.75, more=0.5)


def test_decay_and_passes(B):
    check(B, config("kv4", 2, 8, 2, 400), [333, 48], 3, 3, decay=0.0)
    check(B, config("kv4", 2, 8, 2, 400), [333, 48], 3, 3, decay=0.5, passes=3)


def test_many_rows_of_a_batch(B):
    check(B, config("k8v4", 70, 2, 2, 300, n_recent=17), [(37 * b) % 300 for b in range(70)], 2, 4)


def test_after_a_decode(B):
    """The weights of a decode with its own lse sum to one per query row."""
    rng = np.random.default_rng(5)
    cfg = config("kv4", 3, 8, 2, 600)
    lengths = [600, 411, 5]
    layer, _ = fill(B, cfg, lengths, rng)
    q = torch.from_numpy(rng.standard_normal((3, 8, 128)).astype(np.float16)).cuda()
    out, lse, mass = torch.empty_like(q), torch.empty(3, 8, device="cuda"), B.new_mass(cfg)
    layer.decode_ragged(lengths, q, out, lse, B.new_workspace(cfg))
    layer.attn_mass(lengths, q, lse, mass)
    assert torch.allclose(mass.sum(-1), torch.full((3, 2), 4.0, device="cuda"), rtol=1e-4)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    once = mass.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.attn_mass(lengths, q, lse, mass, decay=0.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(mass, once)
    mass.zero_()
    torch.cuda.synchronize()
    layer.attn_mass(lengths, q, lse, mass, stream=side)
    side.synchronize()
    assert torch.equal(mass, once)


def test_head_subset(B):
    """The record is in the cache's own stream order."""
    rng = np.random.default_rng(6)
    heads, T = [3, 0, 4], 260
    K, V = random_kv(rng, (2, 5, T, 128))
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    q = t(rng.standard_normal((2, 10, 2, 128)).astype(np.float16))
    lse = t((6 + rng.random((2, 10, 2))).astype(np.float32))
    got = []
    for cfg in (config("kv4", 2, 10, 5, 300), config("kv4", 2, 6, 3, 300, kv_heads_total=5, kv_head_index=heads)):
        layer, mass = B.Layer(cfg), B.new_mass(cfg)
        layer.append(0, t(K), t(V))
        layer.attn_mass([T, T - 9], q, lse, mass)
        got.append(mass)
    assert torch.equal(got[0][:, heads], got[1])
