"""The operators in the order a serving loop runs them: a tree of drafted
tokens is verified over the cache, the accepted path is appended, its rows'
attention is recorded, and when the cache is full the groups with the least
weight leave; the next decode attends what is left.  Every step is checked
against 64 bits on the tokens that a plain bookkeeping says are there."""
import numpy as np
import pytest
import torch

from _spec_testutil import attention, cached, config, counts, random_kv
from oracle import kvq_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


@pytest.mark.parametrize("form", ["kv4", "k4v2_hadamard", "innerq4", "nuq", "fp16"])
def test_serving_loop(B, form):
    rng = np.random.default_rng(11)
    batch, hq, hkv, n, cap = 2, 4, 2, 6, 420
    g = hq // hkv
    cfg = config(form, batch, hq, hkv, cap)
    layer, mass = B.Layer(cfg), B.new_mass(cfg)
    tree_ws, evict_ws, ws = B.new_tree_workspace(cfg, n), B.new_evict_workspace(cfg), B.new_workspace(cfg)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    lengths = [300, 260]
    K, V = random_kv(rng, (batch, hkv, 300, 128))
    layer.append_ragged([0, 0], lengths, t(K), t(V))
    # the streams' tokens as the library stores them: (key, value, stored value, quantized?) per position
    def stream(b, h, k, v):
        c = dict(cfg, norm_tokens=lengths[b]) if cfg.get("k_channel_norm") else cfg
        return cached(c, O.build_stream(c, k, v), k.shape[0])
    # tokens that the cache holds, oldest first, in fp16: appended ones are quantized as the window moves, groups of 32 at a time
    hist = {(b, h): (K[b, h, :lengths[b]], V[b, h, :lengths[b]]) for b in range(batch) for h in range(hkv)}
    for step in range(3):
        q = rng.standard_normal((batch, hq, n, 128)).astype(np.float16)
        kd, vd = random_kv(rng, (batch, hkv, n, 128), big=False)
        parents = [[-1, 0, 0, 1, 2, 3], [-1, -1, 0, 1, 2, 4]]
        words = B.tree_mask(parents)
        out, lse = torch.zeros(q.shape, dtype=torch.float16, device="cuda"), torch.zeros(q.shape[:3], device="cuda")
        layer.tree_attn(lengths, t(q), t(kd), t(vd), words.cuda(), out, lse, tree_ws)
        path = [[0, 1, 3], [1, 3]]
        weight = np.zeros((batch, n), np.float32)
        for b in range(batch):
            weight[b, path[b]] = 1.0
        layer.attn_mass(lengths, t(q), lse, mass, t(weight), decay=0.9)
        took = [len(x) for x in path]
        kn, vn = np.zeros((batch, hkv, 3, 128), np.float16), np.zeros((batch, hkv, 3, 128), np.float16)
        for b in range(batch):
            kn[b, :, :took[b]], vn[b, :, :took[b]] = kd[b][:, path[b]], vd[b][:, path[b]]
        if step == 0:  # before anything left, the whole history is the store's
            for b in range(batch):
                for h in range(hkv):
                    k, v, stored, quant = stream(b, h, *hist[b, h])
                    for i in range(n):
                        sees = [j for j in range(n) if words[b, i, 0] >> j & 1]
                        kk, vv = (np.concatenate([a, x[b, h, sees].astype(np.float64)]) for a, x in ((k, kd), (v, vd)))
                        ref, rl, *_ = attention(q[b, h * g:(h + 1) * g, i].astype(np.float64), kk, vv, vv, np.zeros(len(kk), bool), 1 / np.sqrt(128.0))
                        got = out[b, h * g:(h + 1) * g, i].cpu().numpy()
                        assert np.abs(got - ref).max() <= 2e-3 * np.abs(ref).max()
                        assert np.abs(lse[b, h * g:(h + 1) * g, i].cpu().numpy() - rl).max() < 1e-4
        layer.append_ragged(lengths, took, t(kn), t(vn))
        lengths = [a + b for a, b in zip(lengths, took)]
    assert float(mass.min()) >= 0 and float(mass[0, :, lengths[0]:].abs().sum()) == 0
    # what a decode attends before, group by group, and after without the groups that left
    q = t(rng.standard_normal((batch, hq, 128)).astype(np.float16))
    drop = [2, 1]
    source = torch.full((batch, hkv, (cap - 36) // 32), -1, dtype=torch.int32, device="cuda")
    before = layer.buf.clone()
    record = mass.clone()
    after = layer.evict(lengths, drop, mass, mass, source, evict_ws)
    o1, l1 = torch.zeros_like(q), torch.zeros(batch, hq, device="cuda")
    layer.decode_ragged(after, q, o1, l1, ws)
    # the same decode over the cache as it was, without the groups that left: their weight is known from kvq_attn_mass
    old = B.Layer(cfg)
    old.buf.copy_(before)
    o0, l0 = torch.zeros_like(q), torch.zeros(batch, hq, device="cuda")
    old.decode_ragged(lengths, q, o0, l0, ws)
    for j in range(hq):
        one = B.new_mass(cfg)
        qj, lj = torch.zeros_like(q), torch.full_like(l0, -np.inf)
        qj[:, j], lj[:, j] = q[:, j], l0[:, j]
        old.attn_mass(lengths, qj, lj, one)
        for b in range(batch):
            h = j // g
            left = (lengths[b] - 36) // 32 - drop[b]
            kept = source[b, h, :left].tolist()
            gone = sorted(set(range(left + drop[b])) - set(kept))
            lost = sum(float(one[b, h, 4 + 32 * i:36 + 32 * i].double().sum()) for i in gone)
            assert abs(float(l1[b, j]) - (float(l0[b, j]) + np.log1p(-lost))) < 1e-4
            total = record[b, h, 4:4 + 32 * (left + drop[b])].double().view(-1, 32).sum(-1)
            assert float(total[gone].max()) <= float(total[kept].min())
    assert [int((mass[b, 0] != 0).sum()) <= after[b] for b in range(batch)] == [True] * batch
    # and the cache takes further tokens
    kn, vn = random_kv(rng, (batch, hkv, 40, 128), big=False)
    layer.append_ragged(after, [40, 33], t(kn), t(vn))
    layer.decode_ragged([after[0] + 40, after[1] + 33], q, o1, l1, ws)
    torch.cuda.synchronize()
    assert torch.isfinite(o1.float()).all() and torch.isfinite(l1).all()
    assert counts(cfg, after[0])[1] == counts(cfg, lengths[0])[1] - (0 if cfg["k_bits"] == 16 else 64)
