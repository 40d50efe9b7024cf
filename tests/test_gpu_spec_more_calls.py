"""Calls of tree attention, record and eviction that the documentation allows
and the other tests leave out."""
import numpy as np
import pytest
import torch

from _spec_testutil import config, fill, random_kv
from test_gpu_mass import check as check_mass
from test_gpu_tree import check as check_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


@pytest.mark.parametrize("form", ["kv4", "nuq", "innerq4"])
@pytest.mark.parametrize("n", [3, 40])
def test_quantized_tokens_alone(B, form, n):
    """No sinks, no window, no drafted token: rows without an fp16 tile, beside
    an empty one and one that is a window alone."""
    check_tree(B, config(form, 4, 4, 2, 400, n_sink=0, n_recent=0), [96, 0, 320, 31], n, seed=100, mask=None)


@pytest.mark.parametrize("n", [1, 256])
def test_a_batch_of_256(B, n):
    """The largest batch, most rows without a node or a token."""
    lengths = [(53 * b) % 97 if b % 5 == 0 else 0 for b in range(256)]
    nodes = [n if b % 10 == 0 else (b % 3) * (n > 1) for b in range(256)]
    nodes = [m if b % 16 == 0 or m < 3 else 2 for b, m in enumerate(nodes)]
    check_tree(B, config("kv8", 256, 1, 1, 100), lengths, n, nodes=nodes, seed=101)


def test_a_record_of_many_rows(B):
    """Several passes over the keys: 1,300 rows of a KV head, decay once."""
    check_mass(B, config("kv4", 2, 4, 2, 400), [333, 48], 650, 102, weights=True, decay=0.5, more=0.5)
    check_mass(B, config("fp16", 2, 4, 2, 400), [333, 48], 129, 103, weights=True, decay=0.5, more=0.5)


@pytest.mark.parametrize("pairs", [[(4, 4), (2, 8)], [(8, 2), (8, 2)]])
def test_captured_calls_of_mixed_heads(B, pairs):
    """Tree attention, record and eviction of a layer in one graph; the
    captured graph begins with a copy."""
    from bit_kv_cache_07_gb300.mixed import MixedLayer
    rng = np.random.default_rng(104)
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    cfg, n = config("kv4", 2, 4, 2, 500), 5
    k, v = (t(x) for x in random_kv(rng, (2, 2, 500, 128), big=False))
    q = t(rng.standard_normal((2, 4, n, 128)).astype(np.float16))
    kd, vd = (t(x) for x in random_kv(rng, (2, 2, n, 128), big=False))
    words = B.tree_mask([[-1, 0, 1, 1, 0]] * 2).cuda()
    start = [t(rng.random((2, 1 if len(set(pairs)) == 2 else 2, 500)).astype(np.float32)) for _ in set(pairs)]

    def program():
        mixed = MixedLayer(cfg, pairs)
        mixed.append_ragged([0, 0], [500, 300], k, v)
        out, lse, mass = torch.zeros_like(q), torch.zeros(2, 4, n, device="cuda"), mixed.new_mass()
        tws, ews = mixed.new_tree_workspace(n), mixed.new_evict_workspace()

        def run():
            for m, s in zip(mass, start):
                m.copy_(s)
            mixed.tree_attn([500, 300], q, kd, vd, words, out, lse, tws)
            mixed.attn_mass([500, 300], q, lse, mass)
            mixed.evict([500, 300], [3, 1], mass, mass, None, ews)
        torch.cuda.synchronize()
        return run, [out, lse, *mass] + [layer.buf for _, _, layer in mixed.parts]
    run, want = program()
    run()
    torch.cuda.synchronize()
    run, got = program()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


@pytest.mark.parametrize("form", ["kv4", "fp16"])
def test_an_eviction_of_nothing(B, form):
    """No row gives up a group: the record is copied, the cache stays; a
    captured eviction whose first node follows a copy."""
    rng = np.random.default_rng(105)
    cfg = config(form, 3, 2, 2, 400)
    layer, _ = fill(B, cfg, [400, 30, 0], rng)
    before, ws = layer.buf.clone(), B.new_evict_workspace(cfg)
    start = torch.from_numpy(rng.random((3, 2, 400)).astype(np.float32)).cuda()
    mass, out = torch.zeros_like(start), torch.full_like(start, 7.0)
    source = torch.full((3, 2, (400 - 36) // 32), -1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mass.copy_(start)
        layer.evict([400, 30, 0], [0, 0, 0], mass, out, source, ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.buf, before)
    for b, T in enumerate([400, 30, 0]):
        assert torch.equal(out[b, :, :T], start[b, :, :T]) and (out[b, :, T:] == 7.0).all()
        groups = max(0, T - 36) // 32
        assert (source[b, :, :groups].cpu() == torch.arange(groups)).all() and (source[b, :, groups:] == -1).all()


@pytest.mark.parametrize("form", ["k8v4", "fp16"])
def test_evictions_on_two_streams(B, form):
    """Two layers at once, each with its own scratch: the same bytes as alone."""
    rng = np.random.default_rng(106)
    cfg = config(form, 2, 4, 2, 3000)
    jobs = []
    for _ in range(2):
        layer, _ = fill(B, cfg, [3000, 1700], rng)
        record = torch.from_numpy(rng.random((2, 2, 3000)).astype(np.float32)).cuda()
        jobs.append((layer, record, layer.buf.clone(), record.clone(), B.new_evict_workspace(cfg)))
    want = []
    for layer, record, *_, ws in jobs:
        layer.evict([3000, 1700], [40, 11], record, record, None, ws)
        torch.cuda.synchronize()
        want.append((layer.buf.clone(), record.clone()))
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(4):
        for layer, record, buf, start, ws in jobs:
            layer.buf.copy_(buf)
            record.copy_(start)
        torch.cuda.synchronize()
        for (layer, record, *_, ws), st in zip(jobs, streams):
            layer.evict([3000, 1700], [40, 11], record, record, None, ws, stream=st)
        torch.cuda.synchronize()
        for (layer, record, *_), (buf, mass) in zip(jobs, want):
            assert torch.equal(layer.buf, buf) and torch.equal(record, mass)


def test_infinite_records(B):
    """A group's total is the sum in 64 bits: an infinity beside entries whose
    fp32 sum would overflow the other way stays that infinity (equal totals:
    the lower group leaves first), opposite infinities are not a number and
    stay longest."""
    T = 36 + 32 * 6
    cfg = config("kv2", 1, 1, 1, T)
    layer, ws = B.Layer(cfg), B.new_evict_workspace(cfg)
    mass = np.zeros((1, 1, T), np.float32)
    g = mass[0, 0, 4:4 + 192].reshape(6, 32)
    g[0, 0], g[0, 1] = np.inf, -np.inf         # not a number
    g[1, 0], g[1, 8:] = np.inf, -3e38          # +inf
    g[2, 5] = np.inf                           # +inf
    g[3, :] = 3e38                             # finite in 64 bits
    g[4, 3], g[4, 4:20] = -np.inf, 3e38        # -inf
    g[5, :] = 1.0
    gone = [4, 5, 3, 1, 2, 0]                  # in this order
    for E in range(1, 6):
        record = torch.from_numpy(mass).cuda()
        source = torch.full((1, 1, 6), -1, dtype=torch.int32, device="cuda")
        layer.evict([T], [E], record, record, source, ws)
        torch.cuda.synchronize()
        kept = sorted(set(range(6)) - set(gone[:E]))
        assert sorted(source[0, 0, :6 - E].tolist()) == kept, E
