"""The operators of the block cache, as cases to measure: a KV cache in blocks of 32 tokens
shared by many requests, held in 8 bits with one scale for each block and KV head.

plan    block tables, packed offsets and slot maps of a step, from the requests' lengths
append  norms of queries and keys per head, rotation, and the 8-bit store of keys and values
attn    attention of the step's tokens over the blocks: causal, with or without a sliding
        window and first tokens that stay visible

With `own` false, `run` computes them in elementary torch operations on the documented
layout; with `own` true it calls the library.  Both work on the same bytes.
"""
import math
import random

import torch

own = False

D = 128  # head dimension
BLOCK = 32  # tokens of a block
E4M3_MAX = 448.0
E_MIN, E_MAX = -40, 40  # exponents of a block's scale
EPS, THETA = 1e-6, 10000.0


def _case(op, batch, hq, hkv, lo, hi, new, rows, name=None, **more):
    """batch requests that hold lo..hi tokens before the step; `new`: tokens of a request in this step
    (text "mixed": most one, some prompts, some none, some ended); rows: the lengths' own seed."""
    c = dict(op=op, batch=batch, hq=hq, hkv=hkv, lo=lo, hi=hi, new=new, rows=rows)
    if op == "append":
        c.update(norm=True, rotate=True, fused=True)
    if op == "attn":
        c.update(window=0, first=0)
    c.update(more)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decode step of a small batch: latency counts
        _case("plan", 16, 1, 1, 1, 32767, 1, 1, "plan 16 requests, a token each"),
        # continuous batching: prompts arrive, requests end, the others take a token each
        _case("plan", 256, 1, 1, 0, 8191, "mixed", 2, "plan 256 requests, prompts and tokens"),
        # one token of one head at the toy context
        _case("append", 1, 1, 1, 1023, 1023, 1, 3, "append toy token"),
        # a decode step of the 28-on-4-head layer, projections in one buffer
        _case("append", 64, 28, 4, 1, 8191, 1, 4, "append 64 tokens of 28 on 4 heads"),
        # prompts of odd lengths of the 32-on-8-head layer, into partly filled blocks too
        _case("append", 6, 32, 8, 0, 77, 2731, 5, "append prompts of 32 on 8 heads", fused=False),
        # the multi-head layer without norms: four prompts of 4k tokens
        _case("append", 4, 32, 32, 0, 0, 4096, 6, "append 4 x 4k of 32 heads", norm=False),
        # one head at the toy context
        _case("attn", 1, 1, 1, 1024, 1024, 1, 7, "attn toy 1k"),
        # the 32-on-8-head layer's batch at its full context
        _case("attn", 16, 32, 8, 32768, 32768, 1, 8, "attn 16 x 32k of 32 on 8 heads"),
        # a ragged batch of the 28-on-4-head layer
        _case("attn", 64, 28, 4, 100, 8191, 1, 9, "attn 64 ragged to 8k of 28 on 4 heads"),
        # a layer with a sliding window and four first tokens
        _case("attn", 16, 32, 8, 8192, 32768, 1, 10, "attn window 4k of 8k to 32k", window=4096, first=4),
        # multi-head attention, chains of five drafted tokens
        _case("attn", 8, 32, 32, 4000, 4096, 5, 11, "attn 8 x 4k of 32 heads, 5 drafted"),
        # one long context
        _case("attn", 1, 32, 8, 262000, 262144, 1, 12, "attn one context of 256k"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attn", "attn", "attn"])
    rows = rng.randrange(1 << 30)
    if op == "plan":
        return _case("plan", _log_int(rng, 1, 256), 1, 1, 0, _log_int(rng, 40, 32767), rng.choice([1, 1, 5, "mixed"]), rows)
    hkv = rng.choice([1, 2, 4, 8, 32])
    hq = hkv * (rng.choice([1, 2, 3, 4, 7, 8]) if hkv < 32 else 1)
    if op == "append":
        new = rng.choice([1, 1, 2, 5, _log_int(rng, 6, 4096)])
        batch = max(1, min(_log_int(rng, 1, 128), 16000 // new))
        hi = _log_int(rng, 1, 32767 if hkv < 32 else 4096)
        hi = max(1, min(hi, 600000 // (batch * hkv)))
        return _case("append", batch, hq, hkv, 0, hi, new, rows, norm=rng.random() < 0.7, rotate=rng.random() < 0.8, fused=rng.random() < 0.5)
    batch, hi = _log_int(rng, 1, 64), _log_int(rng, 40, 131072)
    hi = max(8, min(hi, 4000000 // (batch * hkv)))
    new = rng.choice([1, 1, 1, 2, 4, rng.randrange(3, 17)])
    window = rng.choice([0, 0, 1, _log_int(rng, 2, 8192)])
    lo = rng.choice([hi, max(new, hi // 2), new])
    return _case("attn", batch, hq, hkv, max(new, lo), max(new, hi), new, rows, window=window, first=rng.choice([0, 4, rng.randrange(1, 100)]) if window else 0)


# ------------------------------------------------------------------ lengths, layout


def _rows(c):
    """(tokens before the step, tokens of the step) of every request, from the case alone."""
    r = random.Random(c["rows"])
    before = [r.randint(c["lo"], c["hi"]) for _ in range(c["batch"])]
    if c["new"] == "mixed":
        new = [r.choice([1] * 12 + [0, -1, r.randint(2, 600)]) for _ in range(c["batch"])]
    else:
        new = [c["new"]] * c["batch"]
    if c["op"] == "attn":  # lengths with the step's tokens
        before = [b - n for b, n in zip(before, new)]
    return before, new


def _blocks(tokens):
    return (tokens + BLOCK - 1) // BLOCK


def _sizes(c):
    """What a user chooses: blocks of the pool, row length of the tables, token slots of a step."""
    before, new = _rows(c)
    after = [b + max(0, n) for b, n in zip(before, new)]
    return dict(before=before, new=new, after=after, n_blocks=sum(_blocks(t) for t in after) + 5, max_blocks=max(1, max(_blocks(t) for t in after)) + 1, n_tokens=max(1, sum(max(0, n) for n in new)))


def _config(c, z):
    return dict(
        batch=c["batch"], n_tokens=z["n_tokens"], n_q_heads=c["hq"], n_kv_heads=c["hkv"], head_dim=D, n_blocks=z["n_blocks"],
        max_blocks=z["max_blocks"], window=c.get("window", 0), n_first=c.get("first", 0), rope_theta=THETA if c.get("rotate", True) else 0.0, norm_eps=EPS)


def _chunks(device):
    """Index [32, 8] of the 16-byte chunks of a block's token rows: chunk c of token t lies at c ^ (t % 8)."""
    t, j = torch.arange(BLOCK, device=device)[:, None], torch.arange(8, device=device)[None]
    return j ^ (t % 8)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _host_step(z):
    """The step's arrays for the cases that start from a plan, on the host."""
    start, unit0, row, pos = [0], [0], [], []
    for b, (l, n) in enumerate(zip(z["before"], z["new"])):
        start.append(start[-1] + n)
        unit0.append(unit0[-1] + (_blocks(l + n) - l // BLOCK if n else 0))
        row += [b] * n
        pos += range(l, l + n)
    return start, unit0, row, pos


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    c, z = case, _sizes(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    st = dict(case=c, z=z, n_blocks=z["n_blocks"])
    ids = torch.randperm(z["n_blocks"], generator=g, device="cuda").to(torch.int32)
    # every request holds blocks from all over the pool, the rest is free
    held = z["before"] if c["op"] == "plan" else z["after"]
    count = torch.tensor([_blocks(t) for t in held], device="cuda")
    first = count.cumsum(0) - count
    col = torch.arange(z["max_blocks"], device="cuda")
    st["block_table"] = torch.where(col < count[:, None], ids[(first[:, None] + col).clamp(max=z["n_blocks"] - 1)], torch.zeros_like(ids[:1]))
    used = int(sum(_blocks(t) for t in held))
    st["free_list"] = torch.cat([ids[used:], torch.zeros(used, dtype=torch.int32, device="cuda")])
    st["free_count"] = _i32([z["n_blocks"] - used])
    st["lens"], st["n_new"] = _i32(z["before"]), _i32(z["new"])
    if c["op"] == "plan":
        N, B = z["n_tokens"], c["batch"]
        st["out"] = dict(
            lens=torch.zeros_like(st["lens"]), free_count=torch.zeros_like(st["free_count"]), start=_i32([0] * (B + 1)), unit0=_i32([0] * (B + 1)),
            token_row=_i32([0] * N), position=_i32([0] * N), slot=_i32([0] * N))
    else:
        start, unit0, row, pos = _host_step(z)
        st["out"] = dict(lens=_i32(z["after"]), free_count=st["free_count"], start=_i32(start), unit0=_i32(unit0), token_row=_i32(row), position=_i32(pos))
        at, rows = st["out"]["position"].long(), st["out"]["token_row"].long()
        st["out"]["slot"] = (st["block_table"][rows, at // BLOCK].long() * BLOCK + at % BLOCK).to(torch.int32)
        _prepare_pool(st, c, z, g)
    if own:
        from bit_kv_cache_07_gb300 import blocks
        st["cfg"] = _config(c, z)
        st["tables"] = blocks.Tables(st["cfg"], block_table=st["block_table"], free_list=st["free_list"], **st["out"])
        if c["op"] != "plan":
            st["layer"] = blocks.Layer(st["cfg"], codes=st["codes"], scales=st["scales"])
            st["workspace"] = blocks.new_workspace(st["cfg"])
    return st


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda")


def _prepare_pool(st, c, z, g):
    """Codes of normal values with a maximum near the type's end, the scale's exponent of the block and head beside them."""
    H, N = c["hkv"], z["n_tokens"]
    codes = torch.empty((z["n_blocks"], H, 2, BLOCK, D), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (H * 2 * BLOCK * D))
    for at in range(0, z["n_blocks"], step):
        part = codes[at:at + step]
        part.copy_((_randn(part.shape, g) * 100).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8))
    st["codes"] = codes
    # exponents around -7: a maximum of 3.5
    n = z["n_blocks"] * H * 2
    room = torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device="cuda")  # padded
    st["scales"] = room[:n].view(z["n_blocks"], H, 2)
    st["scales"].copy_(127 - 7 + torch.randint(-1, 2, st["scales"].shape, generator=g, device="cuda"))
    half = torch.float16
    if c["op"] == "append":
        hq = c["hq"]
        if c["fused"]:  # the three projections' rows in one buffer
            x = _randn((N, hq + 2 * H, D), g).to(half)
            st["q"], st["k"], st["v"] = x[:, :hq], x[:, hq:hq + H], x[:, hq + H:]
        else:
            st["q"], st["k"], st["v"] = (_randn((N, h, D), g).to(half) for h in (hq, H, H))
        st["k"][..., :3] *= 6  # channels that stand out
        st["q_weight"], st["k_weight"] = ((1 + 0.2 * _randn((D,), g)).to(half) if c["norm"] else None for _ in range(2))
        st["q_out"] = torch.zeros((N, hq, D), dtype=half, device="cuda")
    else:
        st["q"] = _randn((N, c["hq"], D), g).to(half)
        st["o"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((N, c["hq"]), device="cuda")


# ------------------------------------------------------------------ one pass


def run(st):
    op, o = st["case"]["op"], st["out"]
    if own:
        if op == "plan":
            st["tables"].plan(st["n_new"], lens=st["lens"], free_count=st["free_count"])
        elif op == "append":
            st["layer"].append(st["tables"], st["k"], st["v"], st["q"], st["q_out"], st["q_weight"], st["k_weight"])
        else:
            st["layer"].attn(st["tables"], st["q"], st["o"], st["lse"], st["workspace"])
    else:
        {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}[op](st)
    if op == "plan":
        return dict(o, block_table=st["block_table"], free_list=st["free_list"])
    if op == "append":
        return dict(q=st["q_out"], codes=st["codes"].view(torch.float8_e4m3fn), scales=st["scales"].view(torch.float8_e8m0fnu))
    return dict(out=st["o"], lse=st["lse"])


def _before(x):
    return x.cumsum(0) - x


def _plain_plan(st):
    o, table, N = st["out"], st["block_table"], st["z"]["n_tokens"]
    B, M = table.shape
    lens, n, free = st["lens"].long(), st["n_new"].long(), st["free_count"].long()
    old, after = (lens + BLOCK - 1) // BLOCK, lens + n.clamp(min=0)
    fits = (n >= 0) & (after <= M * BLOCK)
    need = torch.where(fits, (after + BLOCK - 1) // BLOCK - old, 0)
    back = torch.where(n < 0, old, 0)
    total = free + back.sum()
    granted = fits & ((need == 0) | (need.cumsum(0) <= total)) & (torch.where(fits, n, 0).cumsum(0) <= N)
    n = torch.where(granted, n, torch.where(n < 0, -lens, 0))
    need, took = torch.where(granted, need, 0), n.clamp(min=0)
    end = lens + took
    # the free stack: what was free, then the ended requests' blocks in order
    col = torch.arange(M, device="cuda")
    behind = torch.where(col < back[:, None], free + _before(back)[:, None] + col, st["n_blocks"])
    stack = torch.cat([st["free_list"], table.new_zeros(1)])
    stack[behind.reshape(-1)] = table.reshape(-1)
    st["free_list"].copy_(stack[:-1])
    # new blocks come from its top
    k = _before(need)[:, None] + col - old[:, None]
    new = (col >= old[:, None]) & (col < (old + need)[:, None])
    table.copy_(torch.where(new, st["free_list"][(total - 1 - k).clamp(0, st["n_blocks"] - 1)], table))
    o["lens"].copy_(lens + n)
    o["free_count"].copy_(total - need.sum())
    units = torch.where(took > 0, (end + BLOCK - 1) // BLOCK - lens // BLOCK, 0)
    for name, x in (("start", took), ("unit0", units)):
        o[name][0] = 0
        o[name][1:] = x.cumsum(0)
    i = torch.arange(N, device="cuda")
    row = torch.searchsorted(took.cumsum(0), i, right=True)
    live = row < B
    row = row.clamp(max=B - 1)
    pos = lens[row] + i - _before(took)[row]
    slot = table[row, (pos // BLOCK).clamp(0, M - 1)].long() * BLOCK + pos % BLOCK
    o["token_row"].copy_(torch.where(live, row, -1))
    o["position"].copy_(torch.where(live, pos, 0))
    o["slot"].copy_(torch.where(live, slot, -1))


def _norm_rotate(x, weight, pos, theta):
    """x [N, H, D] in fp32: divided by its root mean square, weighted, pairs (i, i + D/2) rotated."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    if theta:
        turn = pos.double()[:, None] * theta ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        cos, sin = turn.cos().float()[:, None], turn.sin().float()[:, None]
        a, b = x[..., :D // 2], x[..., D // 2:]
        x = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return x


def _exponent(amax):
    """The least e of the range with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax.double() / E4M3_MAX)
    return torch.where(amax > 0, e - (m == 0.5).int(), E_MIN).clamp(E_MIN, E_MAX)


def _plain_append(st):
    c, o = st["case"], st["out"]
    theta = THETA if c["rotate"] else 0.0
    pos, row, slot = o["position"].long(), o["token_row"].long(), o["slot"].long()
    N, H = st["k"].shape[:2]
    st["q_out"].copy_(_norm_rotate(st["q"], st["q_weight"], pos, theta))
    y = torch.stack([_norm_rotate(st["k"], st["k_weight"], pos, theta), st["v"].float()], 2)  # [N, H, 2, D]
    first = (o["lens"] - o["start"].diff()).long()  # tokens before the step
    unit = (o["unit0"].long()[row] + pos // BLOCK - first[row] // BLOCK)
    U = min(N, N // BLOCK + 2 * c["batch"])  # no more blocks are touched
    amax = torch.zeros((U, H, 2), device="cuda").index_reduce_(0, unit, y.abs().amax(-1), "amax")
    e = _exponent(amax)
    # the unit's block and the tokens it held (units that are not there repeat the last token's)
    block, held = (torch.zeros(U, dtype=torch.long, device="cuda") for _ in range(2))
    block[unit] = slot // BLOCK
    held[unit] = torch.where(pos // BLOCK == first[row] // BLOCK, first[row] % BLOCK, 0)
    live = torch.zeros(U, dtype=torch.bool, device="cuda")
    live[unit] = True
    block = torch.where(live, block, slot[-1] // BLOCK)
    twin = torch.where(live, torch.arange(U, device="cuda"), unit[-1])  # units of one block agree
    e, held = e[twin], held[twin]
    was = st["scales"][block].int() - 127
    e = torch.where(held[:, None, None] > 0, torch.maximum(e, was), e)
    # earlier tokens of the block move to the new scale
    codes = st["codes"][block]
    again = (codes.view(torch.float8_e4m3fn).float() * torch.exp2((was - e).float())[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    there = torch.arange(BLOCK, device="cuda") < held[:, None]
    st["codes"][block] = torch.where(there[:, None, None, :, None], again, codes)
    st["scales"][block] = (e + 127).to(torch.uint8)
    code = (y * torch.exp2(-e[unit].float())[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(N, H, 2, 8, 16)
    at = _chunks("cuda")[slot % BLOCK]  # [N, 8]
    st["codes"].view(-1, H, 2, BLOCK, 8, 16)[(slot // BLOCK)[:, None], :, :, (slot % BLOCK)[:, None], at] = code.permute(0, 3, 1, 2, 4)


def _plain_attn(st):
    c, z, o = st["case"], st["z"], st["out"]
    B, H, g, n = c["batch"], c["hkv"], c["hq"] // c["hkv"], c["new"]
    col = torch.arange(st["block_table"].shape[1], device="cuda").expand(B, -1)
    if c["window"]:  # the blocks that hold visible tokens: the first ones, and the window's
        low = ((o["lens"].long() - n - c["window"] + 1) // BLOCK).clamp(min=_blocks(c["first"]))
        wide = torch.arange(_blocks(c["window"] + n) + 1, device="cuda")
        col = torch.cat([col[:, :_blocks(c["first"])], low[:, None] + wide], 1)
    t = (col[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).view(B, 1, 1, 1, -1)
    T = t.shape[-1]
    table = st["block_table"].gather(1, col.clamp(max=st["block_table"].shape[1] - 1)).long()
    kv = st["codes"][table].view(B, -1, H, 2, BLOCK, 8, 16)
    kv = kv.gather(5, _chunks("cuda")[:, :, None].expand(kv.shape))
    kv = kv.view(torch.float8_e4m3fn).view(B, -1, H, 2, BLOCK, D).float()
    kv = kv * torch.exp2(st["scales"][table].float() - 127)[..., None, None]
    k, v = (kv[:, :, :, i].transpose(1, 2).reshape(B, H, 1, T, D) for i in (0, 1))
    # requests of equal numbers of new tokens: [B, H, g, n, D]
    q = st["q"].float().view(B, n, H, g, D).permute(0, 2, 3, 1, 4)
    pos = o["position"].long().view(B, 1, 1, n, 1)
    sees = t <= pos
    if c["window"]:
        sees &= (t > pos - c["window"]) | (t < c["first"])
    s = (q @ k.transpose(3, 4) / math.sqrt(D)).masked_fill(~sees, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = (s - m).exp()
    l = p.sum(-1, keepdim=True)
    st["o"].copy_((p @ v / l).permute(0, 3, 1, 2, 4).reshape(st["o"].shape))
    st["lse"].copy_((m + l.log()).permute(0, 3, 1, 2, 4).reshape(st["lse"].shape))


# ------------------------------------------------------------------ what a pass cannot do without


def _seen(c, length, n):
    """(pairs of a new token and a token that it sees, tokens that any of them sees) of one request."""
    W, F = c["window"] or 1 << 40, c["first"]
    pairs = 0
    for p in range(length - n, length):
        pairs += min(p + 1, W) + min(F, max(0, p + 1 - W))
    low = max(0, length - n - W + 1)
    return pairs, length - low + min(F, low)


def work(case):
    c, z = case, _sizes(case)
    N, B, H, hq = z["n_tokens"], c["batch"], c["hkv"], c["hq"]
    if c["op"] == "plan":
        fresh = sum(_blocks(a) - _blocks(b) for a, b, n in zip(z["after"], z["before"], z["new"]) if n > 0)
        ended = sum(_blocks(b) for b, n in zip(z["before"], z["new"]) if n < 0)
        return {"bytes": 4 * (5 * B + 3 * N + 2 * fresh + 2 * ended), "flops": 0}
    if c["op"] == "append":
        units = _host_step(z)[1][-1]
        return {"bytes": N * D * (2 * (2 * hq + 2 * H) + 2 * H) + 2 * units * H, "flops": 10 * N * D * (hq + 2 * H)}
    seen = [_seen(c, a, c["new"]) for a in z["after"]]
    pairs, tokens = sum(p for p, _ in seen), sum(t for _, t in seen)
    return {"bytes": tokens * H * 2 * D + N * hq * (4 * D + 4) + 2 * H * _blocks(tokens), "flops": 4 * D * hq * pairs}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attn": _exact_attn}[case["op"]](st)


def _exact_plan(st):
    """Request by request on the host."""
    z, B = st["z"], st["case"]["batch"]
    table, stack = st["block_table"].cpu().tolist(), st["free_list"].cpu().tolist()
    M, N = len(table[0]), z["n_tokens"]
    free = int(st["free_count"])
    for b in range(B):
        if z["new"][b] < 0:
            for j in range(_blocks(z["before"][b])):
                stack[free] = table[b][j]
                free += 1
    all_free, asked, asked_tokens = free, 0, 0
    lens, start, unit0, rows, pos, slot = [], [0], [0], [], [], []
    for b in range(B):
        l, n = z["before"][b], z["new"][b]
        took = 0
        if n >= 0 and l + n <= M * BLOCK:
            need = _blocks(l + n) - _blocks(l)
            asked, asked_tokens = asked + need, asked_tokens + n
            if (need == 0 or asked <= all_free) and asked_tokens <= N:
                took = n
                for j in range(_blocks(l), _blocks(l + n)):
                    free -= 1
                    table[b][j] = stack[free]
        lens.append(0 if n < 0 else l + took)
        start.append(start[-1] + took)
        unit0.append(unit0[-1] + (_blocks(l + took) - l // BLOCK if took else 0))
        for p in range(l, l + took):
            rows.append(b)
            pos.append(p)
            slot.append(table[b][p // BLOCK] * BLOCK + p % BLOCK)
    pad = N - len(rows)
    return dict(
        lens=_i32(lens), free_count=_i32([free]), start=_i32(start), unit0=_i32(unit0), token_row=_i32(rows + [-1] * pad),
        position=_i32(pos + [0] * pad), slot=_i32(slot + [-1] * pad), block_table=_i32(table), free_list=_i32(stack))


def _exact_rows(x, weight, pos, rotate):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * weight.double()
    if rotate:
        i = torch.arange(D // 2, device="cuda", dtype=torch.float64)
        angle = pos.double()[:, None] / THETA ** (2 * i / D)
        z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * torch.exp(1j * angle)[:, None]
        x = torch.cat([z.real, z.imag], -1)
    return x


def _exact_append(st):
    """Request by request and block by block; the stored values unrounded."""
    c, z, o = st["case"], st["z"], st["out"]
    pos = o["position"]
    q = _exact_rows(st["q"], st["q_weight"], pos, c["rotate"])
    k, v = _exact_rows(st["k"], st["k_weight"], pos, c["rotate"]), st["v"].double()
    codes = torch.zeros(st["codes"].shape, dtype=torch.float64, device="cuda")
    codes.copy_(st["codes"].view(torch.float8_e4m3fn))
    scales = torch.exp2(st["scales"].double() - 127)
    table, start = st["block_table"].cpu().tolist(), o["start"].cpu().tolist()
    lane = torch.arange(D, device="cuda")
    if sum(_blocks(n + BLOCK) for n in z["new"]) > 6000:
        return None
    for b in range(c["batch"]):
        l, end = z["before"][b], z["after"][b]
        while l < end:
            j, off = l // BLOCK, l % BLOCK
            m = min(BLOCK - off, end - l)
            blk, i = table[b][j], start[b] + l - z["before"][b]
            for side, y in enumerate((k, v)):
                part = y[i:i + m].transpose(0, 1)  # [H, m, D]
                top = part.abs().amax((1, 2))
                e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(E_MIN, E_MAX)
                if off:
                    was = torch.log2(scales[blk, :, side])
                    e = torch.maximum(e, was)
                    codes[blk, :, side, :off] *= torch.exp2(was - e)[:, None, None]
                scales[blk, :, side] = torch.exp2(e)
                for u in range(m):
                    t = off + u
                    codes[blk, :, side, t, (lane // 16 ^ t % 8) * 16 + lane % 16] = part[:, u] * torch.exp2(-e)[:, None]
            l += m
    return dict(q=q, codes=codes, scales=scales)


def _exact_attn(st):
    """Request by request and head by head."""
    c, z, o = st["case"], st["z"], st["out"]
    H, g, n = c["hkv"], c["hq"] // c["hkv"], c["new"]
    if c["batch"] * H > 2100:
        return None
    out, lse = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda"), torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    r = torch.arange(BLOCK, device="cuda")[:, None]
    lane = torch.arange(D, device="cuda")[None]
    place = r * D + (lane // 16 ^ r % 8) * 16 + lane % 16  # byte of a block where (token, channel) lies
    for b in range(c["batch"]):
        L = z["after"][b]
        ids = st["block_table"][b, :_blocks(L)].long()
        t = torch.arange(L, device="cuda")
        p = torch.arange(L - n, L, device="cuda")[:, None]
        hidden = t > p
        if c["window"]:
            hidden |= (p - t >= c["window"]) & (t >= c["first"])
        for h in range(H):
            kv = st["codes"][ids, h].view(len(ids), 2, BLOCK * D)[:, :, place].view(torch.float8_e4m3fn).double()
            kv = kv * torch.exp2(st["scales"][ids, h].double() - 127)[:, :, None, None]
            k, v = kv[:, 0].reshape(-1, D)[:L], kv[:, 1].reshape(-1, D)[:L]
            q = st["q"][b * n:(b + 1) * n, h * g:(h + 1) * g].double()
            s = (torch.einsum("ngd,td->ngt", q, k) / math.sqrt(D)).masked_fill(hidden[:, None], -math.inf)
            lse[b * n:(b + 1) * n, h * g:(h + 1) * g] = torch.logsumexp(s, -1)
            out[b * n:(b + 1) * n, h * g:(h + 1) * g] = torch.softmax(s, -1) @ v
    return dict(out=out, lse=lse)
