"""kvq_block_attn against 64 bits, computed from the stored bytes.

Tolerances, relative to the largest |v| that a row sees (vmax, which bounds every
weighted mean): the weights round to fp16, 2^-11 of each, and their sum of fp32
terms is not rounded so, so a mean moves by at most 2^-11 vmax; weights below
2^-26 of the reference lose more, at most 2^-37 each, nothing at these lengths;
logits are fp32 sums of 128 products, off by at most 2^-20 * sum |q k| scale, with a
factor 2 vmax; and out rounds to fp16, 2^-11 |out|.  lse: the logits' error and
2^-22 |lse|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_kv_cache_07_gb300 import blocks  # noqa: E402
from tests._block_testutil import BLOCK, D, attention, values  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


class Pool:
    """Random codes and scales, requests of given lengths whose blocks lie anywhere."""

    def __init__(self, lens, new, hq, hkv, seed=0, spare=0, n_tokens=None, pad_batch=0, **cfg):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.new, self.hq, self.hkv = lens, new, hq, hkv
        counts = [-(-l // BLOCK) for l in lens]
        B = len(lens) + pad_batch
        N = sum(new) if n_tokens is None else n_tokens
        self.cfg = dict(batch=B, n_tokens=max(1, N), n_q_heads=hq, n_kv_heads=hkv, head_dim=128, n_blocks=max(1, sum(counts)) + spare,
                        max_blocks=max(1, max(counts)))
        self.cfg.update(cfg)
        nb = self.cfg["n_blocks"]
        self.codes = rng.integers(0, 256, (nb, hkv, 2, BLOCK, D), np.uint8)
        self.codes[(self.codes & 127) == 127] = 3
        # mostly moderate codes: a logit's spread of a few
        self.codes = np.where(rng.random(self.codes.shape) < 0.9, (self.codes & 0x80) | rng.integers(0x20, 0x50, self.codes.shape, np.uint8), self.codes).astype(np.uint8)
        self.scales = (127 - 5 + rng.integers(-2, 3, (nb, hkv, 2))).astype(np.uint8)
        ids = rng.permutation(nb)[:sum(counts)]
        self.table = np.zeros((B, self.cfg["max_blocks"]), np.int32)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.q = rng.standard_normal((self.cfg["n_tokens"], hq, D)).astype(np.float16)

    def gpu(self):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        pad = self.cfg["batch"] - len(self.lens)
        start = np.concatenate([[0], np.cumsum(self.new + [0] * pad)]).astype(np.int32)
        t = blocks.Tables(self.cfg, block_table=dev(self.table), lens=dev(np.array(self.lens + [0] * pad, np.int32)), start=dev(start))
        room = torch.zeros(blocks.layout(self.cfg).scales_bytes, dtype=torch.uint8, device="cuda")
        scales = room[:self.scales.size].view(self.scales.shape)
        scales.copy_(dev(self.scales))
        layer = blocks.Layer(self.cfg, codes=dev(self.codes), scales=scales)
        return t, layer, blocks.new_workspace(self.cfg)

    def run(self, times=1):
        t, layer, ws = self.gpu()
        q = torch.from_numpy(self.q).cuda()
        for _ in range(times):
            out = torch.full_like(q, 7.0)
            lse = torch.full(q.shape[:2], 7.0, device="cuda")
            layer.attn(t, q, out, lse, ws)
        assert int(ws[:1024].sum()) == 0  # the counters
        return out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)

    def check(self, out, lse, skip=()):
        kv = values(self.codes, self.scales)
        c, at, g = self.cfg, 0, self.hq // self.hkv
        scale = c.get("softmax_scale") or 1 / np.sqrt(D)
        for b, (l, n) in enumerate(zip(self.lens, self.new)):
            rows = slice(at, at + n)
            at += n
            if b in skip or n == 0:
                continue
            o, s = attention(self.q[rows], kv, self.table[b], l, n, self.hq, self.hkv, c.get("window", 0), c.get("n_first", 0), scale)
            ids = self.table[b, :-(-l // BLOCK)]
            vmax = np.nanmax(np.abs(kv[ids, :, 1]), (0, 2, 3)).repeat(g)[None, :, None]
            kmax = np.nanmax(np.abs(kv[ids, :, 0]).transpose(1, 0, 2, 3).reshape(self.hkv, -1, D), 1).repeat(g, 0)  # [hq, D]
            dz = 2.0**-20 * scale * (np.abs(self.q[rows].astype(float)) * kmax[None]).sum(-1)  # [n, hq]
            bound = 2.0**-11 * vmax + 2 * dz[..., None] * vmax + 2.0**-11 * np.abs(o) + 2.0**-25
            assert (np.abs(out[rows] - o) <= bound).all(), (b, np.max(np.abs(out[rows] - o) / bound))
            assert (np.abs(lse[rows] - s) <= dz + 2.0**-22 * np.abs(s) + 2.0**-22).all(), (b, np.max(np.abs(lse[rows] - s)))
        assert (out[at:] == 7.0).all() and (lse[at:] == 7.0).all()


LENS = [
    ([1], [1]), ([32], [1]), ([33], [1]), ([31, 64, 65, 1], [1, 1, 1, 1]), ([5, 200, 37, 96], [5, 3, 0, 1]),
    ([700], [2]), ([3000, 10], [1, 1]), ([40, 300], [40, 17]), ([257, 90, 513], [1, 64, 33]),
]


@pytest.mark.parametrize("lens,new", LENS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1), (7, 1), (8, 2), (6, 6), (16, 1)])
def test_causal(lens, new, hq, hkv):
    p = Pool(lens, new, hq, hkv, seed=sum(lens) + hq)
    p.check(*p.run())


@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (2, 0), (31, 3), (32, 4), (33, 0), (64, 32), (64, 33), (100, 4), (5, 70),
                                          (256, 1000), (700, 5), (2**31 - 1, 4), (40, 2**31 - 1)])
@pytest.mark.parametrize("lens,new", [LENS[4], LENS[5], LENS[7], ([1, 33, 129, 700], [1, 1, 1, 1])])
def test_window(window, first, lens, new):
    p = Pool(lens, new, 8, 2, seed=window % 1000 + first % 1000, window=window, n_first=first)
    p.check(*p.run())


@pytest.mark.parametrize("n_tokens,batch", [(40, 0), (33, 7), (200, 500), (40, 1000)])
def test_slots_not_in_use(n_tokens, batch):
    """More token slots and more requests than the step has: both are left alone."""
    p = Pool([64, 33, 100], [1, 30, 2], 4, 2, seed=n_tokens, n_tokens=n_tokens, pad_batch=batch)
    p.check(*p.run())


def test_many_requests():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 400, 300)]
    p = Pool(lens, [1] * 300, 4, 2, seed=9)
    p.check(*p.run())


def test_every_range():
    """Long and short requests mixed: segments that span, end and begin CTAs' ranges."""
    lens = [9000, 1, 4000, 31, 33, 2500, 64, 5, 7000]
    p = Pool(lens, [1, 1, 3, 1, 0, 2, 4, 5, 1], 8, 4, seed=2, window=0)
    p.check(*p.run(times=2))


def test_scale_option():
    p = Pool([300, 77], [1, 2], 4, 2, seed=3, softmax_scale=0.3)
    p.check(*p.run())


def test_the_same_bits_every_time():
    p = Pool([5000, 300, 2222], [1, 4, 2], 8, 2, seed=4)
    a, b = p.run(), p.run(times=3)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_spread_logits():
    """Logits that rise along the context by hundreds: the reference moves again and
    again, and keys far below it keep their share."""
    p = Pool([900], [2], 4, 2, seed=6)
    p.codes[:, :, 0] = 0x38  # keys of ones, times the block's scale
    p.scales[:, :, 0] = 127
    for i, blk in enumerate(p.table[0]):
        p.scales[blk, :, 0] = 118 + (i % 14)
    p.q[:] = np.abs(p.q)
    p.check(*p.run())


def test_wide_value_scales():
    """Value scales that differ by tens of octaves between blocks."""
    p = Pool([400, 100], [1, 3], 4, 2, seed=7)
    p.scales[:, :, 1] = np.random.default_rng(1).integers(87, 167, p.scales[:, :, 1].shape)
    kv = values(p.codes, p.scales)
    big = np.abs(kv[:, :, 1]).max()
    assert big > 2.0**40
    p.scales[:, :, 1] = np.where(p.scales[:, :, 1] > 134, 134, p.scales[:, :, 1])  # sums within fp16
    p.check(*p.run())


def test_sink_and_small_rest():
    """One key far above the others: their share, a few percent in all, stays."""
    p = Pool([20000], [1], 2, 1, seed=8)
    p.q[:] = 0
    p.q[..., 0] = 1.0
    p.codes[:, :, 0] = 0
    p.scales[:, :, 0] = 127
    first = p.table[0, 0]
    p.codes[first, 0, 0, 0, 0] = 0x38 + 8 * 6 + 6  # token 0, channel 0: 112 -> 9.9 nats above
    p.check(*p.run())


def test_blocks_marked_as_nan():
    """A marked block makes the rows that see it NaN and no others."""
    p = Pool([300, 300, 300], [1, 1, 6], 4, 2, seed=9, window=64, n_first=2)
    p.scales[p.table[0, 4], 1, 0] = 255  # request 0: behind its window
    p.scales[p.table[1, 9], 0, 1] = 255  # request 1: the last block, values of head 0
    p.scales[p.table[2, 7], 1, 0] = 255  # request 2: tokens 224..255, keys of head 1
    out, lse = p.run()
    p.check(out, lse, skip=(1, 2))
    assert np.isnan(out[1, :2]).all() and np.isfinite(out[1, 2:]).all()
    # the six rows see from 294 - 63 = 231 .. 299 - 63 = 236 on: all see the block
    assert np.isnan(out[2:8, 2:]).all() and np.isfinite(out[2:8, :2]).all() and np.isnan(lse[2:8, 2:]).all()
    q = Pool([300], [6], 4, 2, seed=9, window=40)
    q.scales[q.table[0, 7], 1, 0] = 255  # tokens 224..255; the rows see from 255, 256, .. on
    out, lse = q.run()
    assert np.isnan(out[0, 2:]).all() and np.isfinite(out[1:, :]).all() and np.isfinite(out[:, :2]).all()


def test_block_ids_out_of_range():
    p = Pool([100, 100], [1, 1], 4, 2, seed=10, spare=2)
    p.table[0, 2] = p.cfg["n_blocks"]
    good = p.table[1, 0]
    out, lse = p.run()
    p.table[0, 2] = good
    p.check(out, lse, skip=(0,))
    assert np.isnan(out[0]).all() and np.isnan(lse[0]).all()
    p.table[0, 2] = -7
    out, _ = p.run()
    assert np.isnan(out[0]).all() and np.isfinite(out[1]).all()


def test_lengths_out_of_range_leave_rows_alone():
    p = Pool([100, 64, 50], [1, 1, 1], 4, 2, seed=11)
    t, layer, ws = p.gpu()
    t.lens[0], t.lens[2] = 32 * p.cfg["max_blocks"] + 1, 0
    q = torch.from_numpy(p.q).cuda()
    out = torch.full_like(q, 7.0)
    layer.attn(t, q, out, None, ws)
    o = out.cpu().numpy()
    assert (o[0] == 7.0).all() and (o[2] == 7.0).all() and (o[1] != 7.0).any()


def test_infinite_and_nan_queries():
    p = Pool([200, 90], [3, 1], 4, 2, seed=12)
    p.q[1, 2, 7] = np.nan
    p.q[0, 1, 3] = np.inf
    out, lse = p.run()
    assert np.isnan(out[1, 2]).all() and np.isnan(out[0, 1]).all()
    bad = np.isnan(out).any(-1)
    assert bad.sum() == 2


def test_two_streams_and_shared_tables():
    p = Pool([2000, 300], [2, 1], 8, 2, seed=13)
    t, layer, ws = p.gpu()
    q = torch.from_numpy(p.q).cuda()
    want = torch.zeros_like(q)
    layer.attn(t, q, want, None, ws)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    w = [blocks.new_workspace(p.cfg) for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            layer.attn(t, q, outs[i], None, w[i], stream=s[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_refused():
    p = Pool([64], [1], 4, 2)
    t, layer, ws = p.gpu()
    q = torch.from_numpy(p.q).cuda()
    out = torch.zeros_like(q)
    from bit_kv_cache_07_gb300.binding import KvqError
    with pytest.raises(KvqError):
        layer.attn(t, q, out)
    with pytest.raises(KvqError):
        layer.attn(t, q, out, None, ws[:1024])
    with pytest.raises(KvqError):
        layer.attn(t, q, q, None, ws)
    for bad in (q.float(), q.cpu(), q[:, :3], None):
        with pytest.raises(ValueError):
            layer.attn(t, bad, out, None, ws)
        with pytest.raises(ValueError):
            layer.attn(t, q, bad, None, ws)
    with pytest.raises(ValueError):
        layer.attn(t, q, out, torch.zeros((2, 4), device="cuda"), ws)
    with pytest.raises(ValueError):
        layer.attn(t, q, out, torch.zeros((1, 4), dtype=torch.float16, device="cuda"), ws)
