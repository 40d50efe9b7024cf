"""The block cache over its range: random batches of every kind of segment (whole,
cut, taken by one team, by several rows' passes), full batches, pools past 2^32 bytes,
blocks that requests share, graphs that share a workspace.  Bounds as in
test_gpu_block_attn.py and test_gpu_block_append.py."""
import random

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_kv_cache_07_gb300 import blocks  # noqa: E402
from tests._block_testutil import D, attention, half_step, normed_rotated, values  # noqa: E402
from tests.test_gpu_block_attn import Pool  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


@pytest.mark.parametrize("seed", range(40))
def test_random_batches(seed):
    r = random.Random(seed)
    B = r.choice([1, 2, 5, 17, 64])
    hkv = r.choice([1, 2, 3, 8])
    g = r.choice([1, 2, 3, 4, 7, 8, 12])
    top = r.choice([40, 300, 1500]) if B * hkv * g > 200 else r.choice([40, 700, 6000])
    lens = [r.randint(1, r.choice([40, top])) for _ in range(B)]
    new = [min(l, r.choice([0, 1, 1, 1, 2, 5, r.randint(1, 24)])) for l in lens]
    cfg = {}
    if r.random() < 0.5:
        cfg = dict(window=r.choice([1, 17, 64, 500]), n_first=r.choice([0, 4, 33]))
    p = Pool(lens, new, g * hkv, hkv, seed=seed, n_tokens=max(1, sum(new)) + r.choice([0, 0, 9]), pad_batch=r.choice([0, 3]), **cfg)
    p.check(*p.run())


def test_full_batch():
    """1024 requests: four per thread of the schedule; the first and last hold most."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 70, 1024)]
    lens[0], lens[1023] = 900, 1200
    p = Pool(lens, [1] * 1024, 2, 1, seed=5)
    p.check(*p.run())


def test_every_row_tile_count():
    """17 to 80 rows of a KV head: two and four row tiles side by side, and a second pass."""
    for n in (3, 4, 5, 7, 8, 9, 13, 16, 17, 20):
        p = Pool([700 + n, 150], [n, n], 8, 2, seed=n)
        p.check(*p.run())


def test_one_request_brings_more_than_the_others():
    """A call sized for single tokens in which one request has hundreds of rows."""
    lens, new = [100] * 30 + [900], [1] * 30 + [130]
    p = Pool(lens, new, 8, 2, seed=1)
    p.check(*p.run())


def test_past_32_bits():
    """Blocks whose bytes lie beyond 2^32, in the append and in the attention."""
    H, nb = 8, (1 << 32) // (8 * 8192) + 40
    cfg = dict(batch=2, n_tokens=45, n_q_heads=16, n_kv_heads=H, head_dim=128, n_blocks=nb, max_blocks=3, rope_theta=10000.0, norm_eps=1e-6)
    layer, t = blocks.Layer(cfg), blocks.Tables(cfg)
    top = [nb - 1, nb - 2, nb - 30]
    t.free_list[-3:] = torch.tensor(top[::-1], dtype=torch.int32)  # on top of the stack
    rng = np.random.default_rng(0)
    x = rng.standard_normal((45, 16 + 2 * H, D)).astype(np.float16)
    w = (1 + 0.1 * rng.standard_normal(D)).astype(np.float16)
    g, gw = torch.from_numpy(x).cuda(), torch.from_numpy(w).cuda()
    t.plan(torch.tensor([40, 5], dtype=torch.int32, device="cuda"))
    assert t.block_table[0, :2].tolist() == top[:2] and int(t.block_table[1, 0]) == top[2]
    assert t.slot.max().item() == top[0] * 32 + 31
    q = torch.zeros((45, 16, D), dtype=torch.float16, device="cuda")
    layer.append(t, g[:, 16:16 + H], g[:, 16 + H:], g[:, :16], q, gw, gw)
    out, lse = torch.zeros_like(q), torch.zeros((45, 16), device="cuda")
    layer.attn(t, q, out, lse, blocks.new_workspace(cfg))
    low = layer.codes[:nb - 31]
    assert int(torch.count_nonzero(low.view(-1)[:1 << 30])) == 0 and int(torch.count_nonzero(low.view(-1)[-(1 << 30):])) == 0
    codes, scales = layer.codes[nb - 30:].cpu().numpy(), layer.scales[nb - 30:].cpu().numpy()
    kv = values(codes, scales)
    got, gl = out.cpu().numpy().astype(float), lse.cpu().numpy()
    for b, (l, at, ids) in enumerate(((40, 0, [29, 28]), (5, 40, [0]))):
        k = normed_rotated(x[at:at + l, 16:16 + H], w, range(l), 10000.0)
        held = kv[ids, :, 0].transpose(0, 2, 1, 3).reshape(-1, H, D)[:l]
        unit = 2.0 ** (scales[ids, :, 0].astype(float) - 127).repeat(32, 0)[:l, :, None]
        assert (np.abs(held - k) <= half_step(np.abs(k) / unit) * unit + 2.0**-17 * np.abs(k).max()).all()
        o, s = attention(q.cpu().numpy()[at:at + l], kv, ids, l, l, 16, H)
        vmax = np.abs(kv[ids, :, 1]).max()
        assert (np.abs(got[at:at + l] - o) <= 2.0**-10 * vmax + 2.0**-16 * vmax).all()
        assert (np.abs(gl[at:at + l] - s) <= 2.0**-15).all()


def test_blocks_read_by_several_requests():
    """Requests whose tables begin with the same blocks (read only)."""
    p = Pool([200, 200, 200], [1, 2, 1], 4, 2, seed=4)
    p.table[1, :5], p.table[2, :6] = p.table[0, :5], p.table[0, :6]
    p.check(*p.run())


def test_graphs_that_share_a_workspace():
    a, b = Pool([3000, 200], [1, 3], 8, 2, seed=1), Pool([64, 1000, 5000], [1, 1, 1], 4, 4, seed=2)
    ws = blocks.new_workspace(a.cfg)
    runs = []
    for p in (a, b):
        t, layer, _ = p.gpu()
        q = torch.from_numpy(p.q).cuda()
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.attn(t, q, out, lse, ws)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                layer.attn(t, q, out, lse, ws)
        torch.cuda.current_stream().wait_stream(side)
        runs.append((p, graph, out, lse, t, layer, q))
    for _ in range(5):
        for p, graph, out, lse, *_ in runs:
            out.fill_(7.0)
            lse.fill_(7.0)
            graph.replay()
    for p, graph, out, lse, *_ in runs:
        p.check(out.cpu().numpy().astype(float), lse.cpu().numpy().astype(float))
    assert int(ws[:1024].sum()) == 0


def test_append_and_attention_at_once():
    """Two layers on two streams over one set of tables."""
    p = Pool([500, 70], [1, 2], 8, 2, seed=6, spare=4, rope_theta=10000.0)
    t, layer, ws = p.gpu()
    t.position.copy_(torch.tensor([499, 68, 69], dtype=torch.int32))
    t.unit0.copy_(torch.tensor([0, 1, 2], dtype=torch.int32))
    t.token_row.copy_(torch.tensor([0, 1, 1], dtype=torch.int32))
    other = blocks.Layer(p.cfg)
    other.scales.fill_(127)
    q = torch.from_numpy(p.q).cuda()
    k, v = torch.randn((3, 2, D), device="cuda").half(), torch.randn((3, 2, D), device="cuda").half()
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        layer.attn(t, q, out, lse, ws, stream=s[0])
        other.append(t, k, v, stream=s[1])
    torch.cuda.synchronize()
    p.check(out.cpu().numpy().astype(float), lse.cpu().numpy().astype(float))
    assert int((other.codes != 0).reshape(p.cfg["n_blocks"], -1).any(1).sum()) == 2
