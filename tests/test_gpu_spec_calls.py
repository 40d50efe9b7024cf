"""kvq_tree_attn, kvq_attn_mass and kvq_evict as a serving program calls them:
two streams at once, captured graphs that share a workspace, a budget of SMs,
and tensors that the binding refuses.  Results on other streams, grids of the
same size and replays are the same bits; a smaller grid cuts the work
elsewhere and is compared with the 64-bit formula by test_gpu_tree's bound."""
import numpy as np
import pytest
import torch

from _spec_testutil import config, fill, random_kv
from test_gpu_mass import check as check_mass
from test_gpu_tree import check, tree_masks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


def setup(B, form, lengths, n, seed, g=4, max_tokens=2000):
    """A call of tree attention, then the record: run(stream) and its results."""
    rng = np.random.default_rng(seed)
    batch, hkv = len(lengths), 2
    cfg = config(form, batch, g * hkv, hkv, max_tokens)
    layer, _ = fill(B, cfg, lengths, rng)
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    q = t(rng.standard_normal((batch, g * hkv, n, 128)).astype(np.float16))
    kd, vd = (t(x) for x in random_kv(rng, (batch, hkv, n, 128)))
    words = tree_masks(B, rng, batch, n, [n] * batch).cuda()
    out, lse, mass = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda"), B.new_mass(cfg)
    ws = B.new_tree_workspace(cfg, n)

    def run(stream=None, ws=ws):
        layer.tree_attn(lengths, q, kd, vd, words, out, lse, ws, stream=stream)
        layer.attn_mass(lengths, q, lse, mass, decay=0.0, stream=stream)
    return run, (out, lse, mass), ws


@pytest.mark.parametrize("forms", [("kv4", "kv4"), ("nuq_rope", "fp16"), ("innerq4", "k4v2_hadamard")])
def test_two_streams_at_once(B, forms):
    calls = [setup(B, f, [1900, 700], n, 20 + i) for i, (f, n) in enumerate(zip(forms, (3, 40)))]
    want = []
    for run, got, _ in calls:
        run()
        torch.cuda.synchronize()
        want.append([x.clone() for x in got])
    for _, got, _ in calls:
        for x in got:
            x.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for (run, _, _), st in zip(calls, streams):
            run(stream=st)
    torch.cuda.synchronize()
    for (_, got, _), w in zip(calls, want):
        assert all(torch.equal(x, y) for x, y in zip(got, w))


def test_graphs_that_share_a_workspace(B):
    first, second = setup(B, "kv4", [1900, 5], 3, 30), setup(B, "kv4", [400, 1200], 40, 31)
    ws = max(first[2], second[2], key=lambda w: w.numel())
    graphs, want = [], []
    for run, got, _ in (first, second):
        run(ws=ws)
        torch.cuda.synchronize()
        want.append([x.clone() for x in got])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(ws=ws)
        graphs.append(graph)
        for x in got:
            x.zero_()
    ws.fill_(0xFF)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (_, got, _), w in zip((first, second), want):
        assert all(torch.equal(x, y) for x, y in zip(got, w))


@pytest.mark.parametrize("budget", [1, 7])
@pytest.mark.parametrize("n", [4, 40])
def test_a_budget_of_sms(B, budget, n):
    check(B, config("kv4", 3, 8, 2, 1000, sm_budget=budget), [997, 0, 300], n)


@pytest.mark.parametrize("n", [3, 40])
def test_many_outliers_before_rope(B, n):
    """Eight outliers a vector, pairs that RoPE turns together among them."""
    cfg = config("nuq_rope", 2, 8, 4, 1000, outliers_per_vector=8, position_offset=77)
    check(B, cfg, [997, 333], n)
    check_mass(B, cfg, [997, 333], n, 5)


@pytest.mark.parametrize("form", ["kv4", "fp16"])
def test_the_longest_rows_of_a_workspace_for_more(B, form):
    """Fewer nodes than the workspace was made for, and a call that uses all of max_tokens."""
    run, got, _ = setup(B, form, [2000, 2000], 2, 40)
    big = B.new_tree_workspace(config(form, 2, 8, 2, 2000), 256)
    run()
    torch.cuda.synchronize()
    want = [x.clone() for x in got]
    run(ws=big)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_refused_tensors(B):
    cfg = config("kv4", 1, 4, 2, 300)
    layer = B.Layer(cfg)
    q = torch.zeros(1, 4, 2, 128, dtype=torch.float16, device="cuda")
    kv = torch.zeros(1, 2, 2, 128, dtype=torch.float16, device="cuda")
    words, lse = B.tree_mask([[-1, 0]]).cuda(), torch.zeros(1, 4, 2, device="cuda")
    ws, mass, ews = B.new_tree_workspace(cfg, 2), B.new_mass(cfg), B.new_evict_workspace(cfg)
    strided = torch.zeros(1, 4, 2, 256, dtype=torch.float16, device="cuda")[..., ::2]
    for bad in (dict(q=strided), dict(q=q.float()), dict(out=q.cpu()), dict(kv=kv[:, :1]), dict(words=words.long()), dict(ws=ws.cpu()),
                dict(lse=lse.double())):
        a = dict(q=q, kv=kv, words=words, out=torch.zeros_like(q), lse=lse, ws=ws)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            layer.tree_attn([100], a["q"], a["kv"], a["kv"], a["words"], a["out"], a["lse"], a["ws"])
    with pytest.raises(B.KvqError):  # no workspace, too small a one
        layer.tree_attn([100], q, kv, kv, words, torch.zeros_like(q), lse, None)
    with pytest.raises(B.KvqError):
        layer.tree_attn([100], q, kv, kv, words, torch.zeros_like(q), lse, ws[:4096])
    for bad in (dict(q=strided), dict(lse=lse.half()), dict(mass=mass[:, :1]), dict(mass=mass.cpu()), dict(weight=torch.ones(1, 2))):
        a = dict(q=q, lse=lse, mass=mass, weight=None)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            layer.attn_mass([100], a["q"], a["lse"], a["mass"], a["weight"])
    for bad in (dict(mass=mass.half()), dict(out=mass[:, :1]), dict(source=torch.zeros(1, 2, 3, device="cuda"))):
        a = dict(mass=mass, out=mass, source=None)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            layer.evict([200], [1], a["mass"], a["out"], a["source"], ews)
    with pytest.raises(B.KvqError):  # records that overlap without being the same
        both = torch.zeros(2 * 300 * 2 + 32, device="cuda")
        layer.evict([200], [1], both[:600].view(1, 2, 300), both[32:632].view(1, 2, 300), None, ews)
