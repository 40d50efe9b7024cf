"""Shared helpers of the tests of kvq_tree_attn, kvq_attn_mass and kvq_evict:
configurations, caches filled row by row, and the cached keys and values of a
stream in 64 bits (from the stored bytes that the CPU oracle builds)."""
from __future__ import annotations

import numpy as np

from oracle import kvq_oracle as O

LUT = [-1.5, -0.84375, -0.46875, -0.15625, 0.15625, 0.46875, 0.84375, 1.5]

FORMS = {
    "kv8": dict(k_bits=8, v_bits=8), "k8v4": dict(k_bits=8, v_bits=4), "kv4": dict(k_bits=4, v_bits=4),
    "k4v2": dict(k_bits=4, v_bits=2), "kv2": dict(k_bits=2, v_bits=2), "k2v8": dict(k_bits=2, v_bits=8),
    "k4v2_hadamard": dict(k_bits=4, v_bits=2, v_hadamard=1), "kv4_g32": dict(k_bits=4, v_bits=4, v_group_channels=32),
    "k8v2_g128": dict(k_bits=8, v_bits=2, v_group_channels=128),
    "innerq4": dict(k_bits=4, v_bits=4, k_group_channels=64, hybrid_groups=1, k_channel_norm=1),
    "innerq2": dict(k_bits=2, v_bits=8, k_group_channels=64, hybrid_groups=1),
    "innerq8": dict(k_bits=8, v_bits=2, k_group_channels=64, k_channel_norm=1),
    "nuq": dict(k_bits=3, v_bits=3, outliers_per_vector=2),
    "nuq_hadamard": dict(k_bits=3, v_bits=3, outliers_per_vector=8, v_hadamard=1),
    "nuq_rope": dict(k_bits=3, v_bits=3, outliers_per_vector=1, k_pre_rope=1),
    "kv4_rope": dict(k_bits=4, v_bits=4, k_pre_rope=1, position_offset=1000),
    "fp16": dict(k_bits=16, v_bits=16), "fp16_rope": dict(k_bits=16, v_bits=16, k_pre_rope=1),
}


def config(form, batch, hq, hkv, max_tokens, **kw):
    c = dict(batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, max_tokens=max_tokens, k_group_tokens=32,
             v_group_channels=64, n_sink=4, n_recent=32, v_hadamard=0, k_pre_rope=0, rope_theta=10000.0,
             outliers_per_vector=0, softmax_scale=0.0, split_tokens=0, position_offset=0, k_lut=LUT, v_lut=LUT)
    c.update(FORMS[form])
    c.update(kw)
    return c


def counts(cfg, T):
    """Sinks present, quantized tokens, window tokens (no token: none of each)."""
    return O.layout_counts(cfg, T) if T else (0, 0, 0)


def random_kv(rng, shape, big=True):
    """fp16 keys (three large channels) and heavy-tailed values."""
    k = rng.standard_normal(shape)
    if big:
        k[..., rng.permutation(shape[-1])[:3]] *= 8.0
    return k.astype(np.float16), rng.laplace(size=shape).astype(np.float16)


def f16(x):
    return np.ascontiguousarray(x).view(np.float16).astype(np.float64)


HADAMARD = np.array([[(-1.0) ** bin(i & j).count("1") for j in range(128)] for i in range(128)]) / np.sqrt(128.0)


def dequantized(cfg, store, T):
    """(keys, values, values as stored, quantized flag per token) of a stream
    from its oracle store, [T, 128] in 64 bits by position.  Keys are rotated
    where they were cached before RoPE; `values` are rotated back."""
    S, Nq, W = counts(cfg, T)
    kb, vb = cfg["k_bits"], cfg["v_bits"]
    out = []
    for n, bits in (("k", kb), ("v", vb)):
        x = np.zeros((Nq, 128))
        if Nq:
            code = np.stack([O.unpack_bits(r, 128, bits) for r in store[n + "c"]]).astype(np.float64)
            sc = f16(store[n + "s"]) if bits == 3 else None
            if bits == 3:
                L = np.asarray(cfg[n + "_lut"])
                x = sc[:, :1] + sc[:, 1:] * (L[code.astype(int)] - L[0])
                p = store[n + "_rowptr"]
                for t in range(Nq):
                    x[t, store[n + "_cols"][p[t]:p[t + 1]]] = f16(store[n + "_vals"][p[t]:p[t + 1]])
            else:
                sc = f16(store[n + "s"])  # [groups or tokens, channels or channel groups, 2]
                sc = np.repeat(sc, Nq // sc.shape[0], 0)
                sc = np.repeat(sc, 128 // sc.shape[1], 1)
                x = sc[..., 0] + code * sc[..., 1]
            if n == "k" and cfg.get("k_channel_norm"):
                x = x * store["kn"][None].astype(np.float64)
        sink, win = f16(store[n + "sink"]) if S else np.zeros((0, 128)), f16(store[n + "win"])
        out.append(np.concatenate([sink.reshape(-1, 128), x, win.reshape(-1, 128)])[:T])
    k, stored = out
    if cfg["k_pre_rope"]:
        pos = cfg.get("position_offset", 0) + np.arange(T, dtype=np.float64)[:, None]
        a = pos * np.float64(np.float32(cfg["rope_theta"])) ** (-np.arange(64) / 64.0)
        lo, hi = k[:, :64].copy(), k[:, 64:].copy()
        k = np.concatenate([lo * np.cos(a) - hi * np.sin(a), hi * np.cos(a) + lo * np.sin(a)], 1)
    quant = np.zeros(T, bool)
    quant[S:S + Nq] = True
    v = stored.copy()
    if cfg["v_hadamard"]:
        v[quant] = v[quant] @ HADAMARD
    return k, v, stored, quant


def build_row(cfg, K, V, T):
    """Oracle stores of batch row tokens K, V [Hkv, >= T, 128]."""
    return [O.build_stream(cfg, K[h, :T], V[h, :T]) if T else None for h in range(K.shape[0])]


def cached(cfg, store, T):
    if not T:
        z = np.zeros((0, 128))
        return z, z, z, np.zeros(0, bool)
    return dequantized(cfg, store, T)


def fill(B, cfg, lengths, rng, big=True):
    """A binding.Layer holding lengths[b] random tokens per row, and the
    oracle stores by stream (None for an empty row)."""
    import torch
    hkv, n = cfg["n_kv_heads"], max(max(lengths), 1)
    K, V = random_kv(rng, (cfg["batch"], hkv, n, 128), big)
    layer = B.Layer(cfg)
    if max(lengths):
        layer.append_ragged([0] * cfg["batch"], lengths, torch.from_numpy(K).cuda(), torch.from_numpy(V).cuda())
    stores = []
    for b, T in enumerate(lengths):
        stores += build_row(cfg, K[b], V[b], T)
    return layer, stores


def attention(q, k, v, stored, quant, scale, sees=None):
    """fp64 attention of rows q [r, 128]: (out, lse, sum p |v|, its 2-norm in
    the stored domain of the quantized tokens).  sees [r, tokens] or None."""
    z = scale * (q @ k.T)
    if sees is not None:
        z = np.where(sees, z, -np.inf)
    m = z.max(1, initial=-np.inf)
    m0 = np.where(np.isfinite(m), m, 0.0)
    p = np.exp(z - m0[:, None])
    l = p.sum(1)
    w = p / np.where(l > 0, l, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, m0 + np.log(np.where(l > 0, l, 1.0)), -np.inf)
    spread = w[:, ~quant] @ np.abs(v[~quant])
    rotated = np.linalg.norm(w[:, quant] @ np.abs(stored[quant]), axis=1)
    direct = w[:, quant] @ np.abs(stored[quant])
    return w @ v, lse, spread, rotated, direct
