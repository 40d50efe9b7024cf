"""The operators for speculative decoding and for bounded caches, as cases to measure.

tree   attention of a tree of drafted tokens over the quantized cache and over
       the drafted tokens themselves (each node sees its ancestors)
mass   the attention weight that query rows put on every cached token, added
       to a per-token record of each KV head
evict  the 32-token groups with the least recorded weight leave the cache,
       which is compacted in place

With `own` false, `run` computes them in elementary torch operations on the
layer buffer's documented layout; with `own` true it calls the library.  Both
work on the same bytes: `prepare` quantizes random keys and values itself.
"""
import math

import numpy as np
import torch

own = False

D = 128  # head dimension
GROUP = 32  # tokens of a quantized group
NUQ = [-1.5, -0.84375, -0.46875, -0.15625, 0.15625, 0.46875, 0.84375, 1.5]  # 3-bit level table (exact in fp16)

# (K bits, V bits) and the options of a cache form
FORMS = {
    "kv8": dict(kb=8, vb=8), "k8v4": dict(kb=8, vb=4), "kv4": dict(kb=4, vb=4), "k4v2": dict(kb=4, vb=2),
    "kv2": dict(kb=2, vb=2), "k4v2h": dict(kb=4, vb=2, hadamard=1), "kv4g32": dict(kb=4, vb=4, vgroup=32),
    "innerq": dict(kb=4, vb=4, kgroup=64), "nuq": dict(kb=3, vb=3, outliers=2),
    "nuqrope": dict(kb=3, vb=3, outliers=2, rope=1), "kv4rope": dict(kb=4, vb=4, rope=1),
    "fp16": dict(kb=16, vb=16),
}


def _case(op, form, batch, hq, hkv, tokens, sink, recent, name=None, **more):
    c = dict(op=op, form=form, batch=batch, hq=hq, hkv=hkv, tokens=tokens, sink=sink, recent=recent, ragged=False)
    c.update(more)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one head at the toy context: a short chain of drafted tokens, where latency counts
        _case("tree", "k4v2", 1, 1, 1, 1024, 0, 32, "tree toy chain of 4", nodes=4),
        # multi-head attention (one query head per KV head), a small tree
        _case("tree", "kv4", 8, 32, 32, 4096, 4, 64, "tree mha kv4 16 nodes", nodes=16),
        # grouped-query attention over a long context, 128 query rows per KV head
        _case("tree", "kv4", 8, 32, 8, 32768, 4, 128, "tree gqa kv4 32k 32 nodes", nodes=32),
        # a serving batch: every row its own length and its own tree, rotated 2-bit values
        _case("tree", "k4v2h", 16, 28, 4, 8192, 4, 32, "tree ragged hadamard 21 nodes", nodes=21, ragged=True),
        # long context with non-uniform codes and keys cached before RoPE
        _case("tree", "nuqrope", 1, 32, 32, 65536, 0, 0, "tree nuq rope 64k 8 nodes", nodes=8),
        # the unquantized cache with a large tree, odd sizes
        _case("tree", "fp16", 2, 32, 8, 8191, 0, 0, "tree fp16 63 nodes", nodes=63),
        # one short sequence: latency
        _case("mass", "kv8", 1, 32, 8, 777, 4, 64, "mass short", nodes=1),
        # after every decode step of a long-context batch
        _case("mass", "kv2", 16, 32, 8, 32768, 4, 128, "mass decode kv2 32k", nodes=1),
        # after a verified tree: many rows, of which the accepted ones count
        _case("mass", "innerq", 4, 32, 8, 32768, 4, 32, "mass ragged tree innerq", nodes=17, ragged=True),
        # one sequence gives up a tenth of its groups
        _case("evict", "kv4", 1, 32, 8, 2048, 4, 64, "evict one sequence", share=0.1),
        # a long-context batch gives up a quarter
        _case("evict", "k8v4", 16, 32, 8, 32768, 4, 128, "evict batch k8v4 32k", share=0.25),
        # the unquantized cache, sequences of different lengths
        _case("evict", "fp16", 4, 32, 8, 8192, 4, 64, "evict ragged fp16", share=0.3, ragged=True),
    ]


def draw(rng):
    op = rng.choice(["tree", "tree", "mass", "evict"])
    forms = [f for f in FORMS if op != "evict" or not FORMS[f].get("rope")]
    form = rng.choice(forms)
    hkv = rng.choice([1, 2, 4, 5, 8, 32])
    g = rng.choice([1, 2, 3, 4, 7, 8]) if hkv < 32 else 1
    tokens = int(math.exp(rng.uniform(math.log(1), math.log(32768))))
    batch = max(1, min(rng.choice([1, 2, 3, 8, 16]), (1 << 20) // (tokens * hkv)))
    sink, recent = rng.choice([0, 1, 4]), rng.choice([0, 17, 32, 128])
    c = _case(op, form, batch, g * hkv, hkv, tokens, sink, recent, ragged=rng.random() < 0.4)
    if op == "evict":
        c["share"] = round(rng.uniform(0.02, 0.6), 3)
    else:
        most = max(1, min(64, (1 << 29) // (tokens * batch * g * hkv * 4)))
        c["nodes"] = int(math.exp(rng.uniform(0, math.log(most + 0.99))))
    return c


# ---------------------------------------------------------------- geometry


def _geo(c):
    f = dict(dict(vgroup=64, kgroup=0, hadamard=0, rope=0, outliers=0), **FORMS[c["form"]])
    f["fp16"] = f["kb"] == 16
    f["NS"], f["g"] = c["batch"] * c["hkv"], c["hq"] // c["hkv"]
    f["cap"] = c["tokens"] + 64
    f["S"], f["R"] = (0, 0) if f["fp16"] else (c["sink"], c["recent"])
    f["Q"] = 0 if f["fp16"] else GROUP * max(0, (f["cap"] - f["S"] - f["R"]) // GROUP)
    f["ring"] = f["cap"] if f["fp16"] else f["R"] + GROUP
    return f


def _rows(c):
    """(tokens, nodes, groups to evict) of every batch row: of the case alone."""
    f, B = _geo(c), c["batch"]
    T, n = np.full(B, c["tokens"]), np.full(B, c.get("nodes", 0))
    if c["ragged"]:
        r = np.random.RandomState(c["tokens"] + 7 * B)
        T[1:] = r.randint(max(1, c["tokens"] // 4), c["tokens"] + 1, B - 1)
        n[1:] = r.randint(min(1, c.get("nodes", 0)), c.get("nodes", 0) + 1, B - 1)
    groups = np.maximum(0, (T - c["sink"] - c["recent"]) // GROUP)  # the window rule's whole groups
    quant = np.zeros(B, int) if f["fp16"] else groups * GROUP
    return T, n, quant, groups, (groups * c.get("share", 0.0)).astype(int)


def _layout(c):
    f = _geo(c)
    NS, Q, k = f["NS"], f["Q"], f["outliers"]
    nuq, words = f["kb"] == 3, f["S"] * D * 2
    size = dict(
        k_codes=0 if f["fp16"] else NS * Q * D * f["kb"] // 8,
        k_scales=0 if f["fp16"] else NS * Q * 4 if nuq else NS * Q * 8 if f["kgroup"] else NS * Q // GROUP * D * 4,
        v_codes=0 if f["fp16"] else NS * Q * D * f["vb"] // 8,
        v_scales=0 if f["fp16"] else NS * Q * 4 if nuq else NS * Q * (D // f["vgroup"]) * 4,
        k_sink=NS * words, v_sink=NS * words, k_ring=NS * f["ring"] * D * 2, v_ring=NS * f["ring"] * D * 2,
        k_csr_rowptr=NS * (Q + 1) * 4 if nuq else 0, k_csr_col=NS * Q * k, k_csr_val=NS * Q * k * 2,
        v_csr_rowptr=NS * (Q + 1) * 4 if nuq else 0, v_csr_col=NS * Q * k, v_csr_val=NS * Q * k * 2,
        k_norm=0, rows=2 * 256 * 4)
    at, off = {}, 0
    for name, n in size.items():
        at[name] = (off, n)
        off = (off + n + 255) // 256 * 256
    return at, off


def _views(c, buf):
    """The layer buffer's regions, typed and shaped by stream."""
    f = _geo(c)
    NS, Q, k = f["NS"], f["Q"], f["outliers"]
    at, _ = _layout(c)
    v = {n: buf[o:o + b] for n, (o, b) in at.items()}
    half = torch.float16
    for n, kind in (("k", f["kb"]), ("v", f["vb"])):
        v[n + "_codes"] = v[n + "_codes"].view(NS, Q, -1) if Q else v[n + "_codes"].view(NS, 0, 0)
        v[n + "_scales"] = v[n + "_scales"].view(half).view(NS, Q, -1, 2) if Q and not (n == "k" and kind != 3 and not f["kgroup"]) else \
            v[n + "_scales"].view(half).view(NS, Q // GROUP, D, 2)
        v[n + "_sink"] = v[n + "_sink"].view(half).view(NS, f["S"], D)
        v[n + "_ring"] = v[n + "_ring"].view(half).view(NS, f["ring"], D)
        v[n + "_csr_rowptr"] = v[n + "_csr_rowptr"].view(torch.int32).view(NS, -1)
        v[n + "_csr_col"] = v[n + "_csr_col"].view(NS, Q, k)
        v[n + "_csr_val"] = v[n + "_csr_val"].view(half).view(NS, Q, k)
    return v


def config(c):
    """The kvq_config fields of a case's cache."""
    f = _geo(c)
    return dict(batch=c["batch"], n_q_heads=c["hq"], n_kv_heads=c["hkv"], head_dim=D, max_tokens=f["cap"], k_bits=f["kb"],
                v_bits=f["vb"], k_group_tokens=GROUP, v_group_channels=f["vgroup"], n_sink=c["sink"], n_recent=c["recent"],
                v_hadamard=f["hadamard"], k_pre_rope=f["rope"], rope_theta=10000.0, outliers_per_vector=f["outliers"],
                k_lut=NUQ, v_lut=NUQ, k_group_channels=f["kgroup"])


# ------------------------------------------------------------------ inputs


def _pack(codes, bits):
    """Little-endian bitstream of the codes of each row [..., 128]."""
    per = {8: 1, 4: 2, 2: 4, 3: 8}[bits]
    x = codes.to(torch.int32).view(*codes.shape[:-1], -1, per)
    w = torch.zeros_like(x[..., 0])
    for i in range(per):
        w |= x[..., i] << (bits * i)
    nb = bits * per // 8
    return torch.stack([(w >> (8 * i)) & 255 for i in range(nb)], -1).to(torch.uint8).flatten(-2)


def _uniform(x, bits, dim):
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    sc = (hi - lo) / (2 ** bits - 1)
    code = torch.where(sc > 0, ((x - lo) / sc).round(), torch.zeros_like(x)).clamp(0, 2 ** bits - 1)
    return code, torch.stack([lo, sc], -1).squeeze(dim if dim >= 0 else dim - 1).half()


def _nonuniform(x, k):
    lut = torch.tensor(NUQ, device=x.device)
    col = x.abs().topk(k, -1).indices.sort(-1).values
    out = torch.zeros_like(x, dtype=torch.bool).scatter_(-1, col, True)
    lo = x.masked_fill(out, math.inf).amin(-1, keepdim=True)
    hi = x.masked_fill(out, -math.inf).amax(-1, keepdim=True)
    sc = (hi - lo) / (NUQ[7] - NUQ[0])
    u = (x - lo) / sc + NUQ[0]
    code = torch.bucketize(u, (lut[1:] + lut[:-1]) / 2).masked_fill(out, 0)
    return code, torch.cat([lo, sc], -1).half(), col.to(torch.uint8), x.gather(-1, col).half()


def _fill_cache(c, v, g):
    """Random keys (a few large channels) and values, quantized into the layer buffer row by row."""
    f = _geo(c)
    T, _, quant, _, _ = _rows(c)
    H, S = c["hkv"], f["S"]
    big = torch.rand((H, D), generator=g, device="cuda").argsort(-1)[:, :3]
    gain = torch.ones((H, 1, D), device="cuda").scatter_(2, big[:, None], 8.0)
    for b in range(c["batch"]):
        t, nq, s = int(T[b]), int(quant[b]), slice(b * H, (b + 1) * H)
        x = torch.randn((2, H, t, D), generator=g, device="cuda")
        keys = (x[0] * gain).half()
        vals = (x[1].sign() * torch.expm1(x[1].abs() * 0.7)).half()
        for n, y, bits in (("k", keys, f["kb"]), ("v", vals, f["vb"])):
            v[n + "_sink"][s, :min(S, t)] = y[:, :min(S, t)]
            at = (torch.arange(min(t, S) + nq, t, device="cuda") - S) % f["ring"]
            v[n + "_ring"][s, at] = y[:, min(t, S) + nq:]
            if not nq:
                continue
            z = y[:, S:S + nq].float()
            if n == "v" and f["hadamard"]:
                z = (z @ _hadamard(torch.float32)).half().float()
            if bits == 3:
                code, sc, col, val = _nonuniform(z, f["outliers"])
                v[n + "_scales"][s, :nq] = sc[:, :, None]
                v[n + "_csr_col"][s, :nq], v[n + "_csr_val"][s, :nq] = col, val
            elif n == "k" and not f["kgroup"]:
                code, sc = _uniform(z.view(H, nq // GROUP, GROUP, D), bits, 2)
                v["k_scales"][s, :nq // GROUP] = sc
            else:
                code, sc = _uniform(z.view(H, nq, -1, f["kgroup"] if n == "k" else f["vgroup"]), bits, -1)
                v[n + "_scales"][s, :nq] = sc
            v[n + "_codes"][s, :nq] = _pack(code.reshape(H, nq, D), bits)
    if f["kb"] == 3:
        for n in "kv":
            v[n + "_csr_rowptr"][:] = torch.arange(f["Q"] + 1, device="cuda", dtype=torch.int32) * f["outliers"]


def _tree(c, seed):
    """Random trees: bit j of node i's words is set where j is i or one of its ancestors."""
    B, n = c["batch"], c["nodes"]
    _, count, _, _, _ = _rows(c)
    r = np.random.RandomState(seed % (1 << 31))
    sees = np.zeros((B, n, (n + 31) // 32 * 32), bool)
    for i in range(n):
        up = r.randint(max(-1, i - 9), i, B) if i else np.full(B, -1)
        sees[:, i] = np.where((up >= 0)[:, None], sees[np.arange(B), np.maximum(up, 0)], False)
        sees[:, i, i] = True
        sees[i >= count, i] = False
    words = np.packbits(sees.reshape(B, n, -1, 32), axis=-1, bitorder="little").view(np.uint32)[..., 0]
    return torch.from_numpy(words.view(np.int32).copy()).cuda()


def prepare(case, seed):
    c, f = dict(case), _geo(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    T, count, quant, groups, drop = _rows(c)
    B, H, NS = c["batch"], c["hkv"], f["NS"]
    buf = torch.zeros(_layout(c)[1], dtype=torch.uint8, device="cuda")
    v = _views(c, buf)
    _fill_cache(c, v, g)
    dev = lambda x, t=torch.int64: torch.as_tensor(np.asarray(x), dtype=t, device="cuda")  # noqa: E731
    st = dict(case=c, geo=f, buf=buf, views=v, tokens=[int(x) for x in T], nodes=[int(x) for x in count],
              drop=[int(x) for x in drop], T=dev(T), count=dev(count), quant=dev(quant), groups=dev(groups), E=dev(drop))
    n = c.get("nodes", 0)
    if n:
        st["q"] = torch.randn((B, c["hq"], n, D), generator=g, device="cuda").half()
    if c["op"] == "tree":
        x = torch.randn((2, B, H, n, D), generator=g, device="cuda").half()
        st["k_draft"], st["v_draft"] = x[0].contiguous(), x[1].contiguous()
        st["mask"] = _tree(c, int(seed))
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros(st["q"].shape[:3], device="cuda")
    else:
        t = torch.arange(f["cap"], device="cuda")
        mass = torch.exp(2.0 * torch.randn((B, H, f["cap"]), generator=g, device="cuda")) / c["tokens"]
        st["mass"] = mass * (t < st["T"][:, None, None])
    if c["op"] == "mass":
        # what a decode over the cache alone returns, a little more where drafted tokens took their share
        z = _logits(st, st["q"]).masked_fill(~_valid(st)[0][:, None, None], -math.inf)
        more = torch.rand((B, c["hq"], n), generator=g, device="cuda") * (0.3 if n > 1 else 0.0)
        st["lse"] = (torch.logsumexp(z.double(), -1).float().view(B, c["hq"], n) + more).contiguous()
        # the rows that count: the accepted nodes of a tree (all of a decode's)
        w = (torch.rand((B, n), generator=g, device="cuda") < 0.4).float()
        st["weight"] = w * (torch.arange(n, device="cuda") < st["count"][:, None]) if n > 1 else None
    if c["op"] == "evict":
        st["mass_out"] = torch.zeros_like(st["mass"])
        st["source"] = torch.full((B, H, max(1, (f["cap"] - c["sink"] - c["recent"]) // GROUP)), -1, dtype=torch.int32, device="cuda")
    if own:
        from bit_kv_cache_07_gb300 import binding
        st["cfg"] = binding.make_config(config(c))
        if c["op"] == "tree":
            st["ws"] = binding.new_tree_workspace(st["cfg"], n)
        if c["op"] == "evict":
            st["ws"] = binding.new_evict_workspace(st["cfg"])
    return st


# -------------------------------------------------------------- plain forms


def _hadamard(kind):
    i = torch.arange(D, device="cuda")
    bits = i[:, None] & i[None]
    odd = ((bits[..., None] >> torch.arange(7, device="cuda")) & 1).sum(-1) % 2
    return (1.0 - 2.0 * odd.to(kind)) / math.sqrt(D)


def _codes(packed, bits):
    """Codes [..., 128] of packed rows."""
    if bits == 8:
        return packed
    if bits == 3:
        x = packed.view(*packed.shape[:-1], -1, 3).int()
        w = x[..., 0] | x[..., 1] << 8 | x[..., 2] << 16
        return torch.stack([(w >> s) & 7 for s in (0, 3, 6, 9, 12, 15, 18, 21)], -1).flatten(-2)
    shifts = torch.arange(0, 8, bits, device=packed.device, dtype=torch.uint8)
    return ((packed[..., None] >> shifts) & (2 ** bits - 1)).flatten(-2)


def _quantized(st, n):
    """The dequantized tokens of all streams, in 32 bits: [NS, Qcap, 128] (before any rotation)."""
    f, v = st["geo"], st["views"]
    bits = f["kb"] if n == "k" else f["vb"]
    if not f["Q"]:
        return torch.zeros((f["NS"], 0, D), device="cuda")
    code, sc = _codes(v[n + "_codes"], bits), v[n + "_scales"].float()
    if bits == 3:
        level = torch.tensor(NUQ, device="cuda") - NUQ[0]
        x = sc[..., 0] + sc[..., 1] * level[code.long()]
        return x.scatter(-1, v[n + "_csr_col"].long(), v[n + "_csr_val"].float())
    if n == "k" and not f["kgroup"]:
        x = code.view(f["NS"], -1, GROUP, D).float() * sc[:, :, None, :, 1] + sc[:, :, None, :, 0]
    else:
        x = code.view(*sc.shape[:3], -1).float() * sc[..., 1:] + sc[..., :1]
    return x.reshape(f["NS"], f["Q"], D)


def _valid(st):
    """Which of the slots (sinks, quantized tokens, window ring) hold a token of a batch row, and its position."""
    f, T, nq = st["geo"], st["T"][:, None], st["quant"][:, None]
    a, i, r = (torch.arange(k, device="cuda") for k in (f["S"], f["Q"], f["ring"]))
    first = torch.minimum(T, torch.full_like(T, f["S"])) if f["S"] else torch.zeros_like(T)
    at = f["S"] + nq + (r - nq) % f["ring"]
    ok = torch.cat([(a < first).expand(T.shape[0], -1), i < nq, at < T], 1)
    return ok, torch.cat([a.expand(T.shape[0], -1), (f["S"] + i).expand(T.shape[0], -1), at], 1)


def _keys(st):
    f, v = st["geo"], st["views"]
    k = torch.cat([v["k_sink"].float(), _quantized(st, "k"), v["k_ring"].float()], 1)
    k = k.view(st["case"]["batch"], st["case"]["hkv"], -1, D)
    if f["rope"]:
        pos = _valid(st)[1].double()
        turn = pos[..., None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        co, si = turn.cos().float()[:, None], turn.sin().float()[:, None]
        lo, hi = k[..., :D // 2], k[..., D // 2:]
        k = torch.cat([lo * co - hi * si, hi * co + lo * si], -1)
    return k


def _logits(st, q):
    """Scaled products of the query rows (the heads and nodes of a KV head) with every slot's key."""
    B, H = st["case"]["batch"], st["case"]["hkv"]
    return q.float().view(B, H, -1, D) @ _keys(st).transpose(-1, -2) * (1.0 / math.sqrt(D))


def _plain_tree(st):
    c, f, v = st["case"], st["geo"], st["views"]
    B, H, n = c["batch"], c["hkv"], c["nodes"]
    z = _logits(st, st["q"]).masked_fill(~_valid(st)[0][:, None, None], -math.inf)
    bit = torch.arange(n, device="cuda")
    sees = (st["mask"][..., bit // 32] >> (bit % 32)) & 1
    zd = st["q"].float().view(B, H, -1, D) @ st["k_draft"].float().transpose(-1, -2) * (1.0 / math.sqrt(D))
    zd = zd.view(B, H, f["g"], n, n).masked_fill(sees[:, None, None] == 0, -math.inf).view(B, H, -1, n)
    top = torch.maximum(z.amax(-1), zd.amax(-1))[..., None]
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p, pd = (z - top).exp(), (zd - top).exp()
    total = p.sum(-1, keepdim=True) + pd.sum(-1, keepdim=True)
    a, b = f["S"], f["S"] + f["Q"]
    quantized = p[..., a:b] @ _quantized(st, "v").view(B, H, -1, D)
    if f["hadamard"]:
        quantized = quantized @ _hadamard(torch.float32)
    out = quantized + p[..., :a] @ v["v_sink"].float().view(B, H, -1, D) + p[..., b:] @ v["v_ring"].float().view(B, H, -1, D)
    out = (out + pd @ st["v_draft"].float()) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log()).view(B, c["hq"], n)
    there = (bit < st["count"][:, None])[:, None]
    st["out"].copy_(torch.where(there[..., None], out.view(B, c["hq"], n, D).half(), st["out"]))
    st["lse"].copy_(torch.where(there, lse, st["lse"]))
    return {"out": st["out"], "lse": st["lse"]}


DECAY = 0.875


def _plain_mass(st):
    c, f = st["case"], st["geo"]
    B, H, n = c["batch"], c["hkv"], c["nodes"]
    p = (_logits(st, st["q"]) - st["lse"].view(B, H, -1, 1)).exp()
    if st["weight"] is not None:
        p = p * st["weight"].view(B, 1, 1, n, 1).expand(B, H, f["g"], n, 1).reshape(B, H, -1, 1)
    got = p.sum(2)
    t = torch.arange(f["cap"], device="cuda")
    nq, T = st["quant"][:, None], st["T"][:, None]
    slot = torch.where(t < f["S"] + nq, t, f["S"] + f["Q"] + (t - f["S"]) % f["ring"])
    got = got.gather(-1, slot[:, None].expand(B, H, -1))
    st["mass"].copy_(torch.where((t < T)[:, None], DECAY * st["mass"] + got, st["mass"]))
    return {"mass": st["mass"]}


def _plain_evict(st):
    c, f, v = st["case"], st["geo"], st["views"]
    B, H, S = c["batch"], c["hkv"], c["sink"]
    cap = st["source"].shape[-1]
    ng, E = (x[:, None, None] for x in (st["groups"], st["E"]))
    left = ng - E
    j = torch.arange(cap, device="cuda").expand(B, H, -1)
    whole = torch.zeros((B, H, cap * GROUP), device="cuda")
    have = st["mass"][..., S:S + cap * GROUP]
    whole[..., :have.shape[-1]] = have
    total = whole.view(B, H, cap, GROUP).double().sum(-1).masked_fill(j >= ng, math.inf)
    rank = total.sort(stable=True, dim=-1).indices.argsort(-1)
    gone = (rank < E) & (j < ng)
    # the k-th freed slot below the new end takes the k-th kept group from behind it
    hole, mover = gone & (j < left), ~gone & (j >= left) & (j < ng)
    movers = torch.where(mover, j, cap + j).sort(-1).values
    fill = movers.gather(-1, (hole.long().cumsum(-1) - 1).clamp(min=0))
    source = torch.where(hole, fill, j)
    st["source"].copy_(torch.where(j < left, source, st["source"]))
    source = torch.where(j < left, source, j)  # slots from the new end on stay as they were
    outs = {"source": st["source"]}
    ring = f["ring"]
    if f["fp16"]:
        t = torch.arange(ring, device="cuda").expand(B, H, -1)
        i = t - S
        at = torch.where((i >= 0) & (i < left * GROUP), S + source.gather(-1, (i // GROUP).clamp(0, cap - 1)) * GROUP + i % GROUP, t)
        moved = (i >= left * GROUP) & (t < st["T"][:, None, None] - E * GROUP)
        at = torch.where(moved, t + E * GROUP, at).reshape(f["NS"], ring, 1).expand(-1, -1, D)
        for n in ("k_ring", "v_ring"):
            v[n].copy_(v[n].gather(1, at))
            outs[n] = v[n]
    else:
        flat = source.reshape(f["NS"], -1)[:, :f["Q"] // GROUP]
        for n in ("k_codes", "k_scales", "v_codes", "v_scales", "k_csr_col", "k_csr_val", "v_csr_col", "v_csr_val"):
            if v[n].numel():
                x = v[n].contiguous().view(torch.uint8).view(f["NS"], f["Q"] // GROUP, -1)
                x.copy_(x.gather(1, flat[..., None].expand(x.shape)))
                outs[n] = x  # stored words, moved: equal to the byte
        slot = (torch.arange(ring, device="cuda") + (GROUP * E)) % ring
        slot = slot.expand(B, H, -1).reshape(f["NS"], ring, 1).expand(-1, -1, D)
        for n in ("k_ring", "v_ring"):
            v[n].copy_(v[n].gather(1, slot))
            outs[n] = v[n]
    # the record moves with the tokens
    t = torch.arange(f["cap"], device="cuda").expand(B, H, -1)
    i = t - S
    at = torch.where((i >= 0) & (i < left * GROUP), S + source.gather(-1, (i // GROUP).clamp(0, cap - 1)) * GROUP + i % GROUP, t)
    T = st["T"][:, None, None]
    at = torch.where((i >= left * GROUP) & (t < T - E * GROUP), t + E * GROUP, at)
    moved = torch.where(t < T - E * GROUP, st["mass"].gather(-1, at), torch.zeros((), device="cuda"))
    st["mass_out"].copy_(torch.where(t < T, moved, st["mass_out"]))
    outs["mass_out"] = st["mass_out"]
    return outs


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"tree": _plain_tree, "mass": _plain_mass, "evict": _plain_evict}[op](st)
    from bit_kv_cache_07_gb300 import binding
    if op == "tree":
        binding.kvq_tree_attn(st["cfg"], st["buf"], st["tokens"], st["q"], st["k_draft"], st["v_draft"], st["mask"], st["out"],
                              st["lse"], st["ws"], nodes=st["nodes"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "mass":
        binding.kvq_attn_mass(st["cfg"], st["buf"], st["tokens"], st["q"], st["lse"], st["mass"], weight=st["weight"], decay=DECAY)
        return {"mass": st["mass"]}
    binding.kvq_evict(st["cfg"], st["buf"], st["tokens"], st["drop"], st["mass"], st["mass_out"], st["source"], st["ws"])
    f, v, outs = st["geo"], st["views"], {"source": st["source"], "mass_out": st["mass_out"]}
    for n in ("k_codes", "k_scales", "v_codes", "v_scales", "k_csr_col", "k_csr_val", "v_csr_col", "v_csr_val"):
        if v[n].numel() and not f["fp16"]:
            outs[n] = v[n].view(torch.uint8).view(f["NS"], f["Q"] // GROUP, -1)
    return dict(outs, k_ring=v["k_ring"], v_ring=v["v_ring"])


# -------------------------------------------------------------------- work


def work(case):
    f = _geo(case)
    T, count, quant, groups, drop = (x.astype(float) for x in _rows(case))
    H, g, nuq = case["hkv"], f["g"], f["kb"] == 3
    side = lambda bits, per_token: 0 if bits == 16 else D * bits / 8 + (4 + 3 * f["outliers"] if nuq else per_token)  # noqa: E731
    k_token = side(f["kb"], 8 if f["kgroup"] else D * 4 / GROUP)
    v_token = side(f["vb"], D // f["vgroup"] * 4)
    if case["op"] == "tree":
        read = H * (quant.sum() * (k_token + v_token) + (T - quant).sum() * 4 * D)
        n = count.sum()
        small = n * (H * 4 * D + case["hq"] * (4 * D + 4) + 4 * ((case["nodes"] + 31) // 32))
        pairs = (T * count).sum() * H * g + (count * count).sum() * H * g / 2
        return {"bytes": read + small, "flops": 4.0 * D * pairs}
    if case["op"] == "mass":
        read = H * (quant.sum() * k_token + (T - quant).sum() * 2 * D) + count.sum() * case["hq"] * (2 * D + 4)
        return {"bytes": read + 8 * H * T.sum(), "flops": 2.0 * D * (T * count).sum() * H * g}
    movers = np.where(groups > 0, drop * (1 - drop / np.maximum(groups, 1)), 0)  # kept groups behind the new end, on average
    group_bytes = GROUP * (4 * D if f["fp16"] else k_token + v_token)
    window = (T - (0 if f["fp16"] else f["S"]) - groups * GROUP).clip(0) * (drop > 0) * 4 * D
    return {"bytes": H * (2 * (movers.sum() * group_bytes + window.sum()) + 8 * T.sum() + 4 * (groups - drop).sum()), "flops": 0}


# ------------------------------------------------------------------- exact


def _exact_tokens(c, v, s, T):
    """Keys and values of stream s's T tokens by position, in 64 bits, from the layout's definition."""
    f = _geo(c)
    S = min(f["S"], T)
    nq = 0 if f["fp16"] else GROUP * max(0, (T - f["S"] - f["R"]) // GROUP)
    got = []
    for n, bits in (("k", f["kb"]), ("v", f["vb"])):
        parts = [v[n + "_sink"][s, :S].double()]
        if nq:
            rows = v[n + "_codes"][s, :nq].long()
            stream = ((rows[:, :, None] >> torch.arange(8, device="cuda")) & 1).view(nq, D, bits)
            code = (stream * 2 ** torch.arange(bits, device="cuda")).sum(-1)
            if bits == 3:
                m = v[n + "_scales"][s, :nq, 0].double()
                x = m[:, :1] + m[:, 1:] * (torch.tensor(NUQ, device="cuda", dtype=torch.float64)[code] - NUQ[0])
                x[torch.arange(nq, device="cuda")[:, None], v[n + "_csr_col"][s, :nq].long()] = v[n + "_csr_val"][s, :nq].double()
            elif n == "k" and not f["kgroup"]:
                m = v["k_scales"][s, :nq // GROUP].double().repeat_interleave(GROUP, 0)
                x = m[..., 0] + code * m[..., 1]
            else:
                m = v[n + "_scales"][s, :nq].double()
                m = m.repeat_interleave(D // m.shape[1], 1)
                x = m[..., 0] + code * m[..., 1]
            if n == "v" and f["hadamard"]:
                h = torch.ones((1, 1), dtype=torch.float64, device="cuda")
                for _ in range(7):
                    h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
                x = x @ h / math.sqrt(D)
            parts.append(x)
        where = torch.tensor([(t - f["S"]) % f["ring"] for t in range(S + nq, T)], dtype=torch.long, device="cuda")
        parts.append(v[n + "_ring"][s, where].double())
        got.append(torch.cat(parts))
    k, val = got
    if f["rope"]:
        angle = torch.arange(T, device="cuda", dtype=torch.float64)[:, None] * torch.tensor(
            [10000.0 ** (-2.0 * j / D) for j in range(D // 2)], dtype=torch.float64, device="cuda")
        z = torch.complex(k[:, :D // 2], k[:, D // 2:]) * torch.polar(torch.ones_like(angle), angle)
        k = torch.cat([z.real, z.imag], 1)
    return k, val


def exact(case, seed):
    st = prepare(case, seed)
    c, f, v = st["case"], st["geo"], st["views"]
    H, g, n = c["hkv"], f["g"], c.get("nodes", 0)
    if c["op"] == "evict":
        return _exact_evict(st)
    if c["op"] == "mass":
        mass = st["mass"].double()
        for s in range(f["NS"]):
            b, h = divmod(s, H)
            k, _ = _exact_tokens(c, v, s, st["tokens"][b])
            z = st["q"][b, h * g:(h + 1) * g].double() @ k.T / math.sqrt(D)
            p = (z - st["lse"][b, h * g:(h + 1) * g].double()[..., None]).exp()
            if st["weight"] is not None:
                p = p * st["weight"][b].double()[None, :, None]
            mass[b, h, :st["tokens"][b]] = DECAY * mass[b, h, :st["tokens"][b]] + p.sum((0, 1))
        return {"mass": mass}
    out, lse = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda"), torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    for s in range(f["NS"]):
        b, h = divmod(s, H)
        m = st["nodes"][b]
        k, val = _exact_tokens(c, v, s, st["tokens"][b])
        k, val = torch.cat([k, st["k_draft"][b, h, :m].double()]), torch.cat([val, st["v_draft"][b, h, :m].double()])
        words = st["mask"][b, :m].cpu().numpy().view(np.uint32)
        sees = [[j for j in range(m) if words[i, j // 32] >> np.uint32(j % 32) & 1] for i in range(m)]
        allowed = torch.ones((m, k.shape[0]), dtype=torch.bool)
        allowed[:, st["tokens"][b]:] = False
        for i, js in enumerate(sees):
            allowed[i, [st["tokens"][b] + j for j in js]] = True
        z = st["q"][b, h * g:(h + 1) * g, :m].double() @ k.T / math.sqrt(D)
        z = z.masked_fill(~allowed.cuda(), -math.inf)
        lse[b, h * g:(h + 1) * g, :m] = torch.logsumexp(z, -1)
        out[b, h * g:(h + 1) * g, :m] = torch.softmax(z, -1) @ val
    return {"out": out, "lse": lse}


def _exact_evict(st):
    """The surviving groups' places and the record, group by group on the host; the moved words have no 64-bit value."""
    c, f = st["case"], st["geo"]
    S = c["sink"]
    mass, source = st["mass"].double().cpu().numpy(), st["source"].cpu().numpy()
    out = st["mass_out"].double().cpu().numpy()
    for b in range(c["batch"]):
        T, E = st["tokens"][b], st["drop"][b]
        ng = max(0, (T - S - c["recent"]) // GROUP)
        for h in range(c["hkv"]):
            total = [math.fsum(mass[b, h, S + GROUP * j:S + GROUP * (j + 1)]) for j in range(ng)]
            gone = set(sorted(range(ng), key=lambda j: (total[j], j))[:E])
            place = list(range(ng - E))
            behind = [j for j in range(ng - E, ng) if j not in gone]
            for j in sorted(j for j in gone if j < ng - E):
                place[j] = behind.pop(0)
            source[b, h, :ng - E] = place
            took = [mass[b, h, :min(S, T)]] + [mass[b, h, S + GROUP * j:S + GROUP * (j + 1)] for j in place]
            took = np.concatenate(took + [mass[b, h, S + GROUP * ng:T]])
            out[b, h, :T] = 0.0
            out[b, h, :len(took)] = took
    outs = {n: None for n in ("k_codes", "k_scales", "v_codes", "v_scales", "k_csr_col", "k_csr_val", "v_csr_col", "v_csr_val")
            if not f["fp16"] and st["views"][n].numel()}
    return dict(outs, k_ring=None, v_ring=None, source=source, mass_out=out)
