"""The record over channels so wide that a query times a channel's scale passes
fp16's range, for row counts on both sides of the choice between its kernels.

Tolerance: as test_gpu_mass, (e^E - 1 + 2^-16 + n 2^-24) of the sum and 2^-23 of
the entry, with E = 2^-20 scale sum |q k| (it covers the fp32 rounding of the
logit and of its difference to the log-sum-exp, 2^-23 of their size).  The
exponential is fp32 and flushes below its smallest normal number: 2^-126 per
weight, absolute (logits here lie up to 264,000 apart)."""
import numpy as np
import pytest
import torch

from _spec_testutil import build_row, cached, config, random_kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


def check_mass(B, cfg, lengths, K, V, q, more=0.0):
    """One call of the record over a cache of K, V [B, Hkv, T, 128] with rows q
    [B, Hq, n, 128], from an empty record.  more: added to the logits' error."""
    batch, hq, n = q.shape[:3]
    hkv, cap = cfg["n_kv_heads"], cfg["max_tokens"]
    g = hq // hkv
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    layer, mass = B.Layer(cfg), B.new_mass(cfg)
    layer.append_ragged([0] * batch, lengths, t(K), t(V))
    scale, want, lse = 1 / np.sqrt(128.0), {}, np.zeros((batch, hq, n), np.float32)
    for b, T in enumerate(lengths):
        for h, store in enumerate(build_row(cfg, K[b], V[b], T)):
            k = cached(cfg, store, T)[0]
            qs = q[b, h * g:(h + 1) * g].astype(np.float64)
            z, size = scale * (qs @ k.T), scale * (np.abs(qs) @ np.abs(k).T)
            m = z.max(-1, keepdims=True)
            rows = (m[..., 0] + np.log(np.exp(z - m).sum(-1))).astype(np.float32)
            lse[b, h * g:(h + 1) * g] = rows
            p = np.exp(z - rows.astype(np.float64)[..., None])
            want[b, h] = p.sum((0, 1)), 2.0 ** -20 * np.where(p > 0, size, 0).max() + more
    layer.attn_mass(lengths, t(q), t(lse), mass)
    torch.cuda.synchronize()
    got = mass.cpu().numpy()
    for (b, h), (ref, E) in want.items():
        bound = (np.expm1(E) + 2.0 ** -16 + g * n * 2.0 ** -24) * ref + 2.0 ** -23 * ref + g * n * 2.0 ** -126
        x = got[b, h, :lengths[b]]
        assert np.isfinite(x).all() and (np.abs(x - ref) <= bound).all(), (b, h, np.max(np.abs(x - ref) / bound))
        assert (got[b, h, lengths[b]:] == 0).all()


@pytest.mark.parametrize("form", ["kv2", "innerq4"])
@pytest.mark.parametrize("g,n", [(1, 1), (3, 1), (2, 4), (3, 3)])
def test_a_query_times_a_wide_channel(B, form, g, n):
    """Channel 0 holds 60,000 or its negative, the queries 25 there: logits of
    +- 132,000, of which the softmax sees the equal larger ones."""
    rng = np.random.default_rng(70)
    lengths, hkv = [400, 77], 2
    cfg = config(form, 2, hkv * g, hkv, 400)
    K, V = random_kv(rng, (2, hkv, 400, 128), big=False)
    K[..., 0] = np.where(rng.random(K.shape[:-1]) < 0.5, -60000.0, 60000.0)
    q = (0.5 * rng.standard_normal((2, hkv * g, n, 128))).astype(np.float16)
    q[..., 0] = 25.0
    check_mass(B, cfg, lengths, K, V, q)


@pytest.mark.parametrize("form", ["fp16", "kv4"])
@pytest.mark.parametrize("g,n", [(3, 1), (3, 4), (4, 8), (5, 13)])
def test_keys_of_minus_infinity(B, form, g, n):
    """Cached fp16 keys that no query attends (-inf where every query is
    positive): their weight is zero, whatever number of rows meets them and
    whether all of them count."""
    rng = np.random.default_rng(71)
    T, hkv = 500, 2
    cfg = config(form, 1, hkv * g, hkv, T, n_recent=100)
    K, V = random_kv(rng, (1, hkv, T, 128), big=False)
    gone = np.r_[1, 3, T - 90:T - 60, T - 1] if form == "kv4" else np.r_[1, 3, 40:70, 200, T - 1]  # sinks and window; anywhere
    q = rng.standard_normal((1, hkv * g, n, 128)).astype(np.float16)
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    K[:, :, gone, 0] = -np.inf
    q[..., 0] = np.abs(q[..., 0]) + np.float16(0.25)
    check_mass(B, cfg, [T], K, V, q)
    # rows that do not count beside the others
    layer, lse = B.Layer(cfg), torch.full((1, hkv * g, n), 6.0, device="cuda")
    layer.append(0, t(K), t(V))
    weight = torch.ones(1, n, device="cuda")
    weight[0, n // 2:] = 0.0
    got, want = B.new_mass(cfg), B.new_mass(cfg)
    layer.attn_mass([T], t(q), lse, got, weight)
    if n > 1:
        layer.attn_mass([T], t(q[:, :, :n // 2]), lse[:, :, :n // 2].contiguous(), want)
    torch.cuda.synchronize()
    # both within e^E - 1 + 2^-16 of the sum, E <= 2^-20 * 16 (sum |q k| scale of the finite keys)
    assert torch.allclose(got, want, rtol=2.0 ** -14, atol=0.0)
    assert (got[0, :, torch.from_numpy(gone).cuda()] == 0).all()
