"""Tree attention of rows whose weights span a wide range, and what the second
fp16 part of the weights is worth, against attention in 64 bits.

Tolerances, elementwise.  The output rounds to fp16 once, 2^-11 |out| (2^-25
below fp16's normal range).  Logits carry E = 2^-20 scale sum |q k| (22-bit
keys, fp32 accumulation over 128 products) and weights change by e^E - 1,
numerator and denominator: 2 E.  A weight enters in two fp16 parts: 2^-22 of
itself, and no finer than 2^-31 of the largest weight of its row: together with
the fp32 exponential (2^-22) below 2^-20 of itself.  The output is accumulated in
fp32 by products over 16 keys, once for each part of the weights: 2 ceil(n / 16)
steps over n keys, and each may cut the running sum by its last place, 2^-23 (the
instruction does not promise to round): (n + 30) 2^-26 of sum p |v| with the
drafted keys' own.  Values round to fp16 unless they are cached as that: 2^-11."""
import numpy as np
import pytest
import torch

from _spec_testutil import attention, build_row, cached, config, random_kv
from test_gpu_tree import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


def exact(cfg, store, T, q, kd, vd, sees):
    """(out, sum p |v|, sum |v|, largest E) of rows q [n, 128] in 64 bits."""
    k, v, stored, quant = cached(cfg, store, T)
    k, v = np.concatenate([k, kd]), np.concatenate([v, vd])
    quant = np.concatenate([quant, np.zeros(len(kd), bool)])
    scale = 1 / np.sqrt(128.0)
    see = np.concatenate([np.ones((len(q), T), bool), sees], 1)
    out, _, a, _, b = attention(q, k, v, v, quant, scale, see)
    z = scale * (np.abs(q) @ np.abs(k).T)
    return out, a + b, np.abs(v).sum(0), 2.0 ** -20 * np.where(see, z, 0).max(1)


@pytest.mark.parametrize("form", ["fp16", "kv4"])
@pytest.mark.parametrize("n", [5, 20])
@pytest.mark.parametrize("gap", [12.0, 18.0])
def test_a_dominant_first_token(B, form, n, gap):
    """The first token's logit lies `gap` nats above 20,000 others, its value is
    zero: the others, below a thousandth of the weight, are the output.  One
    CTA walks them all."""
    rng = np.random.default_rng(60)
    T = 20000
    cfg = config(form, 1, 1, 1, T, n_sink=0, n_recent=0, sm_budget=1)
    K = (0.4 * rng.standard_normal((1, T, 128))).astype(np.float16)
    V = (1.0 + 0.1 * rng.random((1, T, 128))).astype(np.float16)
    K[0, 0], V[0, 0] = gap / np.sqrt(128.0), 0.0
    q = (1.0 + 0.1 * rng.standard_normal((1, 1, n, 128))).astype(np.float16)
    kd, vd = (0.4 * rng.standard_normal((1, 1, n, 128))).astype(np.float16), np.ones((1, 1, n, 128), np.float16)
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    layer = B.Layer(cfg)
    layer.append(0, t(K[None]), t(V[None]))
    words = B.tree_mask([list(range(-1, n - 1))])
    out = torch.zeros(1, 1, n, 128, dtype=torch.float16, device="cuda")
    layer.tree_attn([T], t(q), t(kd), t(vd), words.cuda(), out, None, B.new_tree_workspace(cfg, n))
    got = out.cpu().numpy()[0, 0].astype(np.float64)
    store = build_row(cfg, K, V, T)[0]
    ref, spread, whole, E = exact(cfg, store, T, q[0, 0].astype(np.float64), kd[0, 0].astype(np.float64),
                                  vd[0, 0].astype(np.float64), bits(words, n)[0])
    values = 0.0 if form == "fp16" else 2.0 ** -11
    bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2.0 ** -20 + (T + n + 30) * 2.0 ** -26 + values + 2 * E[:, None]) * spread + 2.0 ** -31 * whole
    assert (bound < 0.04 * ref).all()  # (losing a sixth of what lies 18 nats below is 4.5 %)
    assert (np.abs(got - ref) <= bound).all(), np.max(np.abs(got - ref) / bound)


@pytest.mark.parametrize("n", [5, 20])
def test_weights_keep_their_second_part(B, n):
    """Values cached as fp16 that nearly cancel: rounding the weights to one fp16
    part would show, in the same bound, in channels whose sum is small."""
    rng = np.random.default_rng(61)
    lengths, hkv = [3, 40, 300], 2
    cfg = config("fp16", 3, 2, hkv, 300)
    K, V = random_kv(rng, (3, hkv, 300, 128), big=False)
    q = rng.standard_normal((3, hkv, n, 128)).astype(np.float16)
    kd, vd = random_kv(rng, (3, hkv, n, 128), big=False)
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    layer = B.Layer(cfg)
    layer.append_ragged([0] * 3, lengths, t(K), t(V))
    words = B.tree_mask([list(range(-1, n - 1))] * 3)
    out = torch.zeros(q.shape, dtype=torch.float16, device="cuda")
    layer.tree_attn(lengths, t(q), t(kd), t(vd), words.cuda(), out, None, B.new_tree_workspace(cfg, n))
    got = out.cpu().numpy().astype(np.float64)
    one_part = 0.0
    for b, T in enumerate(lengths):
        for h, store in enumerate(build_row(cfg, K[b], V[b], T)):
            qs, sees = q[b, h].astype(np.float64), bits(words, n)[b]
            args = kd[b, h].astype(np.float64), vd[b, h].astype(np.float64)
            ref, spread, whole, E = exact(cfg, store, T, qs, *args, sees)
            bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2.0 ** -20 + (T + n + 30) * 2.0 ** -26 + 2 * E[:, None]) * spread + 2.0 ** -31 * whole
            assert (np.abs(got[b, h] - ref) <= bound).all(), (b, h, np.max(np.abs(got[b, h] - ref) / bound))
            # the same with weights in one part, in the oracle
            k, v, _, _ = cached(cfg, store, T)
            z = qs @ np.concatenate([k, args[0]]).T / np.sqrt(128.0)
            p = np.exp(z - z.max(1, keepdims=True)) * np.concatenate([np.ones((n, T), bool), sees], 1)
            o = p.astype(np.float16).astype(np.float64) @ np.concatenate([v, args[1]]) / p.sum(1, keepdims=True)
            one_part = max(one_part, np.max(np.abs(o.astype(np.float16) - ref) / bound))
    assert one_part > 2.0


@pytest.mark.parametrize("form", ["fp16", "k8v4"])
@pytest.mark.parametrize("n", [7, 20])
@pytest.mark.parametrize("jump", [0.0, 130.0])
def test_logits_that_grow(B, form, n, jump):
    """Rows whose logits rise or fall steadily along the cache, each at its own
    rate, from flat to 60 nats over it, some with a step of `jump` nats
    half-way (past fp32's range of the weights before it): references move
    often, for some rows of a warp and not for others."""
    rng = np.random.default_rng(62)
    T = 3000
    cfg = config(form, 1, 1, 1, T, n_sink=0, n_recent=0, sm_budget=1)
    K = (0.3 * rng.standard_normal((1, T, 128))).astype(np.float16)
    V = (1.0 + rng.random((1, T, 128))).astype(np.float16)
    K[0, :, 0] = np.linspace(0.0, 60.0, T)
    K[0, :, 1] = np.where(np.arange(T) < T // 2, 0.0, jump)
    q = (0.3 * rng.standard_normal((1, 1, n, 128))).astype(np.float16)
    q[0, 0, :, 0] = np.linspace(-1.0, 1.0, n) * np.sqrt(128.0)
    q[0, 0, :, 1] = np.where(np.arange(n) % 3 == 0, np.sqrt(128.0), 0.0)
    kd, vd = (0.3 * rng.standard_normal((1, 1, n, 128))).astype(np.float16), np.ones((1, 1, n, 128), np.float16)
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    layer = B.Layer(cfg)
    layer.append(0, t(K[None]), t(V[None]))
    words = B.tree_mask([list(range(-1, n - 1))])
    out = torch.zeros(1, 1, n, 128, dtype=torch.float16, device="cuda")
    layer.tree_attn([T], t(q), t(kd), t(vd), words.cuda(), out, None, B.new_tree_workspace(cfg, n))
    got = out.cpu().numpy()[0, 0].astype(np.float64)
    store = build_row(cfg, K, V, T)[0]
    ref, spread, whole, E = exact(cfg, store, T, q[0, 0].astype(np.float64), kd[0, 0].astype(np.float64),
                                  vd[0, 0].astype(np.float64), bits(words, n)[0])
    values = 0.0 if form == "fp16" else 2.0 ** -11
    # a move multiplies the sums so far by a rounded power of two (2^-22), at most once a tile of 96 keys
    moves = 2.0 ** -22 * (T // 96 + 2)
    bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2.0 ** -20 + moves + (T + n + 30) * 2.0 ** -26 + values + 2 * E[:, None]) * spread + 2.0 ** -31 * whole
    assert (bound < 0.02 * ref).all()
    assert (np.abs(got - ref) <= bound).all(), np.max(np.abs(got - ref) / bound)
