"""kvq_block_append against 64 bits: norm, rotation, scales, codes, tokens that move
to a larger scale, and what has to stay as it was.

Tolerances.  The kernel computes y in fp32: a mean of 128 squares, one reciprocal
square root, two products and a rotation, each with relative errors of a few 2^-24
of the largest of the pair, and sines of an absolute error below 2^-20 (angle 2^-24
included): |dy| <= 2^-18 * |pair| is safe for all of it.  A code is then off by at
most half a step of e4m3 at y (and where y + dy crosses to the next step, no more
than that plus dy); q_out by half a step of fp16, 2^-11 |y|, plus dy."""
import random

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_kv_cache_07_gb300 import blocks  # noqa: E402
from tests._block_testutil import BLOCK, D, EPS, Plan, exponent, half_step, normed_rotated, values  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


class Cache:
    """A layer and its tables on the GPU beside the model: what every token's row should be."""

    def __init__(self, batch, n_tokens, hq, hkv, n_blocks, max_blocks, seed=0, **cfg):
        self.cfg = dict(batch=batch, n_tokens=n_tokens, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, n_blocks=n_blocks,
                        max_blocks=max_blocks, rope_theta=10000.0, norm_eps=EPS)
        self.cfg.update(cfg)
        self.rng = np.random.default_rng(seed)
        self.plan, self.t, self.layer = Plan(batch, n_tokens, n_blocks, max_blocks), blocks.Tables(self.cfg), blocks.Layer(self.cfg)
        self.want = {}  # (request, head, side) -> rows in 64 bits
        self.exp = {}   # (block, head, side) -> exponent
        self.moves = {}  # rows that moved to a larger scale: how often

    def inputs(self, big=1.0):
        N, hq, hkv = self.cfg["n_tokens"], self.cfg["n_q_heads"], self.cfg["n_kv_heads"]
        x = self.rng.standard_normal((N, hq + 2 * hkv, D)) * big
        x[:, hq:hq + hkv, :3] *= 8
        return x.astype(np.float16)

    def weights(self):
        return [(1 + 0.3 * self.rng.standard_normal(D)).astype(np.float16) for _ in range(2)]

    def append(self, new, x, wq, wk, fused=True, queries=True, stream=None):
        c, N = self.cfg, self.cfg["n_tokens"]
        hq, hkv = c["n_q_heads"], c["n_kv_heads"]
        dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.plan.step(new)
        self.t.plan(torch.tensor(new, dtype=torch.int32, device="cuda"))
        if fused:
            g = dev(x)
            q, k, v = g[:, :hq], g[:, hq:hq + hkv], g[:, hq + hkv:]
        else:
            q, k, v = dev(x[:, :hq]), dev(x[:, hq:hq + hkv]), dev(x[:, hq + hkv:])
        out = torch.full((N, hq, D), 7.0, dtype=torch.float16, device="cuda") if queries else None
        self.layer.append(self.t, k, v, q if queries else None, out, dev(wq) if queries else None, dev(wk), stream)
        self.model(new, x, wk)
        used = self.plan.start[-1]
        if queries:
            got = out.cpu().numpy()
            assert (got[used:] == 7.0).all()
            y = normed_rotated(x[:used, :hq], wq, self.plan.pos[:used], c["rope_theta"])
            pair = np.hypot(y[..., :64], y[..., 64:])
            dy = 2.0**-18 * np.concatenate([pair, pair], -1)
            assert (np.abs(got[:used] - y) <= 2.0**-11 * np.abs(y) + 2.0**-25 + dy).all()
        return out

    def model(self, new, x, wk):
        c, p = self.cfg, self.plan
        hq, hkv = c["n_q_heads"], c["n_kv_heads"]
        for b in range(c["batch"]):
            i0, i1 = p.start[b], p.start[b + 1]
            if new[b] < 0:
                for key in [k for k in self.want if k[0] == b]:
                    del self.want[key]
            if i0 == i1:
                continue
            k = normed_rotated(x[i0:i1, hq:hq + hkv], wk, p.pos[i0:i1], c["rope_theta"])
            v = x[i0:i1, hq + hkv:].astype(np.float64)
            for side, y in enumerate((k, v)):
                for h in range(hkv):
                    rows = self.want.setdefault((b, h, side), [])
                    before = len(rows)
                    rows.extend(y[:, h])
                    for j in range(before // BLOCK, -(-len(rows) // BLOCK)):
                        old = max(0, before - j * BLOCK)
                        top = np.abs(np.array(rows[j * BLOCK + old:(j + 1) * BLOCK])).max()
                        key = (int(p.table[b, j]), h, side)
                        if not old:
                            self.exp.pop(key, None)
                        e = self.exp.get(key, -40)
                        near = top * (1 + 2.0**-17)
                        # the exponents that the kernel may take, a maximum next to a border allowing two
                        self.exp[key] = max(e, exponent(top * (1 - 2.0**-17)))
                        self.exp[key + ("up",)] = max(e, exponent(near))
                        if old and self.exp[key] > e:
                            self.moves[key] = self.moves.get(key, 0) + 1

    def check(self):
        codes, scales = self.layer.codes.cpu().numpy(), self.layer.scales.cpu().numpy()
        assert ((codes & 127) != 127).all()  # no code is a NaN
        kv = values(codes, scales)
        for (b, h, side), rows in self.want.items():
            y = np.array(rows)
            for j in range(-(-len(rows) // BLOCK)):
                blk = int(self.plan.table[b, j])
                key = (blk, h, side)
                e = int(scales[blk, h, side]) - 127
                assert e in (self.exp[key], self.exp[key + ("up",)]), (e, self.exp[key])
                part = y[j * BLOCK:(j + 1) * BLOCK]
                got = kv[blk, h, side, :len(part)]
                pair = np.hypot(part[..., :64], part[..., 64:])
                dy = 2.0**-18 * np.concatenate([pair, pair], -1) * (side == 0)
                unit = 2.0**e
                bound = half_step(np.abs(part) / unit) * unit + dy
                # a row that moved was rounded again, by half of the smallest step, each time
                bound = bound + self.moves.get(key, 0) * 2.0**-10 * unit
                assert (np.abs(got - part) <= bound * (1 + 1e-9)).all(), (b, h, side, j, np.max(np.abs(got - part) / bound))


CASES = [
    # batch, hq, hkv, steps of new tokens; the first rows of a block, its middle, its end
    (1, 1, 1, [[1], [1], [30], [1], [40]]),
    (3, 4, 2, [[5, 0, 33], [1, 1, 1], [1, 64, 1], [31, 31, 30], [2, -1, 2], [1, 3, 1]]),
    (2, 7, 1, [[100, 31], [1, 1], [4, 4], [200, 1]]),
    (5, 8, 8, [[1, 2, 3, 4, 5], [4, 4, 4, 4, 4], [0, 0, 0, 0, 9]]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("norm,theta,fused", [(True, 10000.0, True), (True, 0.0, False), (False, 500000.0, False), (False, 0.0, True)])
@pytest.mark.parametrize("few", [True, False])  # one warp per block, eight
def test_steps(case, norm, theta, fused, few):
    batch, hq, hkv, steps = CASES[case]
    most = max(sum(max(0, n) for n in s) for s in steps)
    n_tokens = most if not few else min(most, 4 * batch)
    if few:
        steps = [[min(n, n_tokens // batch) for n in s] for s in steps]
    else:
        n_tokens = max(n_tokens, 4 * batch + 1)
    c = Cache(batch, n_tokens, hq, hkv, 60, 14, seed=case, rope_theta=theta)
    for i, new in enumerate(steps):
        x = c.inputs(big=[1.0, 4.0, 0.25, 16.0, 1.0, 64.0][i % 6])  # scales that grow inside a block
        wq, wk = c.weights() if norm else (None, None)
        c.append(new, x, wq, wk, fused, queries=(i + case) % 3 != 2)
        c.check()


def test_many_tokens_by_one_warp():
    """A call sized for single tokens in which one request brings them all."""
    c = Cache(20, 80, 2, 2, 30, 12, seed=5)
    for new in ([0] * 7 + [77] + [0] * 12, [0] * 7 + [70] + [3] + [0] * 11):
        c.append(new, c.inputs(), *c.weights())
        c.check()


def test_far_positions():
    """Positions past 2^20: the angle keeps its digits."""
    c = Cache(1, 3, 4, 2, 3, 1 << 20, seed=1)
    start = 32 * ((1 << 20) - 1) + 30  # the last block of the longest row
    c.t.lens.fill_(start + 2)
    c.t.start.copy_(torch.tensor([0, 2]))
    c.t.unit0.copy_(torch.tensor([0, 1]))
    c.t.position.copy_(torch.tensor([start, start + 1, 0]))
    c.t.token_row.copy_(torch.tensor([0, 0, -1]))
    c.t.block_table[0, -1] = 2
    x = c.inputs()
    dev = torch.from_numpy(x).cuda()
    wq, wk = (torch.from_numpy(w).cuda() for w in c.weights())
    out = torch.zeros((3, 4, D), dtype=torch.float16, device="cuda")
    c.layer.append(c.t, dev[:, 4:6], dev[:, 6:], dev[:, :4], out, wq, wk)
    y = normed_rotated(x[:2, :4], wq.cpu().numpy(), [start, start + 1], 10000.0)
    pair = np.hypot(y[..., :64], y[..., 64:])
    # (the reference's own angle: a product and a power of 2^25 * 2^-53 relative)
    assert (np.abs(out.cpu().numpy()[:2] - y) <= 2.0**-11 * np.abs(y) + 2.0**-17 * np.concatenate([pair, pair], -1)).all()
    k = normed_rotated(x[:2, 4:6], wk.cpu().numpy(), [start, start + 1], 10000.0)
    scales = c.layer.scales.cpu().numpy()
    got = values(c.layer.codes.cpu().numpy(), scales)[2, :, 0, 30:].transpose(1, 0, 2)
    unit = 2.0 ** (scales[2, :, 0].astype(float) - 127)[None, :, None]
    assert (np.abs(got - k) <= half_step(np.abs(k) / unit) * unit + 2.0**-17 * np.abs(k).max()).all()


def test_large_calls_give_the_bytes_of_small_ones():
    """Several heads per CTA and per warp (rows asked for more than the ring's depth
    ahead) against the same tokens request by request: no sum or maximum reaches over a
    head's block, so the bytes are the same.  The large call's queries lie in place."""
    sizes, hq, hkv = [2731, 3000, 3269], 24, 12
    N = sum(sizes)
    x = torch.from_numpy(np.random.default_rng(11).standard_normal((N, hq + 2 * hkv, D)).astype(np.float16)).cuda()
    w = torch.from_numpy((1 + 0.3 * np.random.default_rng(12).standard_normal((2, D))).astype(np.float16)).cuda()
    k, v = x[:, hq:hq + hkv], x[:, hq + hkv:]

    def cache(batch, n):
        cfg = dict(batch=batch, n_tokens=n, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, n_blocks=300, max_blocks=110,
                   rope_theta=10000.0, norm_eps=EPS)
        return blocks.Tables(cfg), blocks.Layer(cfg)

    t, layer = cache(3, N)
    t.plan(torch.tensor(sizes, dtype=torch.int32, device="cuda"))
    q = x[:, :hq].contiguous()
    layer.append(t, k, v, q, q, w[0], w[1])
    at = 0
    for b, n in enumerate(sizes):
        t1, one = cache(1, n)
        t1.plan(torch.tensor([n], dtype=torch.int32, device="cuda"))
        out = torch.zeros((n, hq, D), dtype=torch.float16, device="cuda")
        rows = slice(at, at + n)
        one.append(t1, k[rows], v[rows], x[rows, :hq], out, w[0], w[1])
        assert torch.equal(out, q[rows])
        used = -(-n // BLOCK)
        ids, ids1 = t.block_table[b, :used].long(), t1.block_table[0, :used].long()
        assert torch.equal(layer.scales[ids], one.scales[ids1])
        tail = n % BLOCK or BLOCK
        assert torch.equal(layer.codes[ids[:-1]], one.codes[ids1[:-1]])
        assert torch.equal(layer.codes[ids[-1], :, :, :tail], one.codes[ids1[-1], :, :, :tail])
        at += n


@pytest.mark.parametrize("batch", [31, 32, 33, 65])
def test_requests_around_a_warp(batch):
    """The search for a block's request takes one step up to 32 requests and two beyond."""
    rng = random.Random(batch)
    new = [rng.choice([0, 1, 5, 40]) for _ in range(batch)]
    new[0], new[-1] = 0, 33
    c = Cache(batch, sum(new) + 3, 2, 1, 3 * batch, 4, seed=batch)
    for step in (new, [1] * batch):
        if sum(step) <= c.cfg["n_tokens"]:
            c.append(step, c.inputs(), *c.weights())
            c.check()


def test_queries_in_place():
    c = Cache(2, 8, 4, 2, 8, 4, seed=3)
    x = c.inputs()
    wq, wk = c.weights()
    apart = c.append([5, 2], x, wq, wk, fused=False)
    q = torch.from_numpy(np.ascontiguousarray(x[:, :4])).cuda()
    k, v = (torch.from_numpy(np.ascontiguousarray(x[:, i:i + 2])).cuda() for i in (4, 6))
    codes = c.layer.codes.clone()
    c.layer.append(c.t, k, v, q, q, torch.from_numpy(wq).cuda(), torch.from_numpy(wk).cuda())
    assert torch.equal(q[:7], apart[:7]) and torch.equal(q[7], torch.from_numpy(x[7, :4]).cuda())
    assert torch.equal(codes, c.layer.codes)  # the same tokens again: the same bytes


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("few", [True, False])
def test_not_finite(bad, few):
    """A block and side with such a token is marked, its codes stay numbers; other
    heads, sides and blocks are as without it; the block is well again for its next owner."""
    n_tokens = 8 if few else 80
    c = Cache(2, n_tokens, 2, 2, 6, 3, seed=4, norm_eps=0.0)
    x = c.inputs()
    good = Cache(2, n_tokens, 2, 2, 6, 3, seed=4, norm_eps=0.0)
    y = x.copy()
    y[1, 2 + 1, 5] = bad   # key of head 1, token 1 of request 0
    y[3, 4 + 0, 100] = bad  # value of head 0, token 3
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    for cache, z in ((c, y), (good, x)):
        cache.t.plan(torch.tensor([4, 2], dtype=torch.int32, device="cuda"))
        g = dev(z)
        cache.layer.append(cache.t, g[:, 2:4], g[:, 4:])
    s, ref = c.layer.scales.cpu().numpy(), good.layer.scales.cpu().numpy()
    blk = int(c.t.block_table[0, 0])
    marked = np.zeros_like(s, bool)
    marked[blk, 1, 0] = marked[blk, 0, 1] = True
    assert (s[marked] == 255).all() and (s[~marked] == ref[~marked]).all()
    a, b = c.layer.codes.cpu().numpy(), good.layer.codes.cpu().numpy()
    assert ((a & 127) != 127).all() and np.array_equal(a[~marked], b[~marked])
    c.t.plan(torch.tensor([1, 1], dtype=torch.int32, device="cuda"))
    c.layer.append(c.t, g[:, 2:4], g[:, 4:])
    assert (c.layer.scales.cpu().numpy()[marked] == 255).all()  # it stays with the block's tokens
    c.t.plan(torch.tensor([-1, -1], dtype=torch.int32, device="cuda"))
    c.t.plan(torch.tensor([4, 4], dtype=torch.int32, device="cuda"))
    c.layer.append(c.t, g[:, 2:4], g[:, 4:])
    assert (c.layer.scales.cpu().numpy()[blk] != 255).all()


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("what", ["key", "weight", "zero row"])
def test_not_finite_after_the_norm(what, few):
    """A norm that is not finite (a key, a weight, a row of zeros with eps 0) marks the
    block's keys; codes stay numbers, values as they are."""
    n_tokens = 8 if few else 80
    c = Cache(2, n_tokens, 2, 2, 6, 3, seed=4, norm_eps=0.0)
    x = c.inputs()
    wq, wk = c.weights()
    if what == "key":
        x[1, 2, 5] = np.inf
    elif what == "weight":
        wk[70] = np.nan
    else:
        x[1, 2] = 0
    g, gw = torch.from_numpy(x).cuda(), torch.from_numpy(wk).cuda()
    c.t.plan(torch.tensor([4, 3], dtype=torch.int32, device="cuda"))
    c.layer.append(c.t, g[:, 2:4], g[:, 4:], k_weight=gw)
    s, codes = c.layer.scales.cpu().numpy(), c.layer.codes.cpu().numpy()
    assert ((codes & 127) != 127).all()
    a, b = int(c.t.block_table[0, 0]), int(c.t.block_table[1, 0])
    assert s[a, 0, 0] == 255 and (s[[a, b], :, 1] != 255).all()
    assert (s[b, :, 0] == 255).all() if what == "weight" else (s[b, :, 0] != 255).all() and s[a, 1, 0] != 255


def test_tables_that_no_plan_writes_are_left_out():
    """Sums of touched blocks far out of range: nothing is written anywhere."""
    c = Cache(3, 40, 2, 2, 6, 3, seed=9)
    g = torch.from_numpy(c.inputs()).cuda()
    c.t.plan(torch.tensor([10, 10, 10], dtype=torch.int32, device="cuda"))
    before = c.layer.codes.clone()
    for unit0 in ([-(2**31), 1, 2, 3], [-(2**27), -(2**27) + 1, 2**30, 2**31 - 1], [0, 0, 0, 2**31 - 1], [5, 5, 5, 9], [7, 3, 1, 0]):
        c.t.unit0.copy_(torch.tensor(unit0, dtype=torch.int32))
        c.layer.append(c.t, g[:, 2:4], g[:, 4:])
    torch.cuda.synchronize()
    changed = (c.layer.codes != before).reshape(6, -1).any(1).nonzero().reshape(-1).tolist()
    assert set(changed) <= {int(c.t.block_table[b, 0]) for b in range(3)}


def test_values_at_the_ends_of_the_range():
    """Zeros, the smallest and largest fp16 numbers, one of each sign."""
    c = Cache(3, 6, 1, 1, 5, 2, seed=6, rope_theta=0.0)
    x = np.zeros((6, 3, D), np.float16)
    x[2, 1:, 0], x[2, 1:, 1] = 65504, -65504
    x[4, 1:, 0], x[4, 1:, 1] = 2.0**-24, -(2.0**-24)
    c.append([2, 2, 2], x, None, None)
    c.check()
    assert sorted(set(c.layer.scales.cpu().numpy()[[int(c.plan.table[b, 0]) for b in range(3)]].reshape(-1).tolist())) == [87, 127 - 32, 127 + 8]


def test_ids_and_lengths_out_of_range_are_left_out():
    c = Cache(4, 8, 2, 2, 6, 3, seed=7)
    x = c.inputs()
    g = torch.from_numpy(x).cuda()
    c.t.plan(torch.tensor([2, 2, 2, 2], dtype=torch.int32, device="cuda"))
    c.t.block_table[0, 0], c.t.block_table[1, 0] = -1, 6
    c.t.lens[2] = 97
    before = c.layer.codes.clone()
    c.layer.append(c.t, g[:, 2:4], g[:, 4:])
    changed = (c.layer.codes != before).reshape(6, -1).any(1).nonzero().reshape(-1).tolist()
    assert changed == [int(c.t.block_table[3, 0])]


def test_other_slots_stay():
    """Bytes of tokens that the step does not bring, of blocks that it does not touch."""
    r = random.Random(3)
    c = Cache(3, 12, 2, 2, 9, 3, seed=8)
    c.append([12, 0, 0], c.inputs(), None, None)
    c.layer.codes.copy_(torch.randint(0, 126, c.layer.codes.shape, dtype=torch.uint8, device="cuda"))
    c.layer.scales.fill_(127 + 30)  # larger than any new maximum: nothing moves
    before, s = c.layer.codes.clone(), c.layer.scales.clone()
    g = torch.from_numpy(c.inputs()).cuda()
    c.plan.step([1, 2, 0])
    c.t.plan(torch.tensor([1, 2, 0], dtype=torch.int32, device="cuda"))
    c.layer.append(c.t, g[:, 2:4], g[:, 4:])
    rows = (c.layer.codes != before).any(-1).any(1).any(1)  # [block, token]
    touched = {(sl // 32, sl % 32) for sl in c.plan.slot[:3]}
    assert {tuple(i) for i in rows.nonzero().tolist()} <= touched
    new = int(c.plan.table[1, 0])
    keep = [i for i in range(9) if i != new]
    assert torch.equal(c.layer.scales[keep], s[keep]) and r


def test_refused_tensors():
    c = Cache(2, 4, 4, 2, 4, 2)
    h = dict(dtype=torch.float16, device="cuda")
    k, q = torch.zeros((4, 2, D), **h), torch.zeros((4, 4, D), **h)
    bad = [torch.zeros((4, 2, D), device="cuda"), torch.zeros((4, 2, D), dtype=torch.float16), torch.zeros((3, 2, D), **h),
           torch.zeros((4, 2, 256), **h)[..., ::2], torch.zeros((2, 4, D), **h).transpose(0, 1), None]
    for x in bad:
        with pytest.raises(ValueError):
            c.layer.append(c.t, x, k)
        with pytest.raises(ValueError):
            c.layer.append(c.t, k, x)
    for args in ((q, None), (None, q), (q, torch.zeros((4, 8, D), **h)[:, ::2]), (q, torch.zeros((4, 6, D), **h)[:, :4])):
        with pytest.raises(ValueError):
            c.layer.append(c.t, k, k.clone(), *args)
    with pytest.raises(ValueError):
        c.layer.append(c.t, k, k.clone(), q, q, torch.zeros(127, **h))
    other = blocks.Layer(dict(c.cfg, n_blocks=5))
    with pytest.raises(ValueError):
        other.append(c.t, k, k.clone())
    with pytest.raises(ValueError):
        blocks.Layer(c.cfg, scales=torch.zeros((4, 2, 2), dtype=torch.uint8, device="cuda")[:, :, :1])
    odd = dict(c.cfg, n_blocks=3)
    with pytest.raises(ValueError):  # 12 bytes: the storage must be padded to 16
        blocks.Layer(odd, scales=torch.zeros((3, 2, 2), dtype=torch.uint8, device="cuda"))
