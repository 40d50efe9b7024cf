"""kvq_evict on the GPU against a plain group-by-group eviction of the layer
buffer's bytes (moves are exact: every byte is compared, the ones that must
stay among them), for every cache form without pre-RoPE keys, in place and
into another record, with ties, zeros, infinities and NaN in the record."""
import math

import numpy as np
import pytest
import torch

from _spec_testutil import FORMS, config, counts, fill

pytestmark = pytest.mark.gpu
EVICT = sorted(f for f in FORMS if not FORMS[f].get("k_pre_rope"))


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


def groups_of(cfg, T):
    return max(0, T - cfg["n_sink"] - cfg["n_recent"]) // 32


def total_of(m):
    m = m.astype(np.float64)
    if np.isnan(m).any():
        return math.inf, 1
    t = math.fsum(m) if np.isfinite(m).all() else float(np.sum(m))
    return (math.inf, 1) if math.isnan(t) else (t, 0)


def plan(cfg, mass, T, E):
    """Where the groups that stay come from, for one stream."""
    S, n = cfg["n_sink"], groups_of(cfg, T)
    order = sorted(range(n), key=lambda j: (*total_of(mass[S + 32 * j:S + 32 * j + 32]), j))
    gone = set(order[:E])
    left = n - E
    place = list(range(left))
    behind = iter(j for j in range(left, n) if j not in gone)
    for j in range(left):
        if j in gone:
            place[j] = next(behind)
    return place


def expected(B, layer, cfg, lengths, drop, mass):
    """(layer bytes, record, source) after a plain eviction."""
    buf = layer.buf.cpu().numpy().copy()
    lay, NS, hkv = layer.layout, cfg["batch"] * cfg["n_kv_heads"], cfg["n_kv_heads"]
    out = mass.copy()
    cap = max(0, cfg["max_tokens"] - cfg["n_sink"] - cfg["n_recent"]) // 32
    source = np.full((cfg["batch"], hkv, cap), -7, np.int32)
    fp16 = cfg["k_bits"] == 16
    view = {}
    for name in B.REGIONS:
        r = getattr(lay, name)
        if r.bytes and not name.endswith("rowptr") and name not in ("rows", "k_norm"):
            view[name] = buf[r.offset:r.offset + r.bytes].reshape(NS, -1)
    for s in range(NS):
        b, h = divmod(s, hkv)
        T, E = lengths[b], drop[b]
        n, S = groups_of(cfg, T), cfg["n_sink"]
        left = n - E
        place = plan(cfg, mass[b, h], T, E)
        source[b, h, :left] = place
        old = mass[b, h].copy()
        kept = np.concatenate([old[:min(S, T)]] + [old[S + 32 * j:S + 32 * j + 32] for j in place] + [old[min(S, T) + 32 * n if n else min(S, T):T]])
        out[b, h, :T] = 0
        out[b, h, :len(kept)] = kept
        if E == 0:
            continue
        for name, v in view.items():
            row = v[s].copy()
            if fp16:
                tok = row.reshape(-1, 256)
                want = tok.copy()
                for j, src in enumerate(place):
                    want[S + 32 * j:S + 32 * j + 32] = tok[S + 32 * src:S + 32 * src + 32]
                want[S + 32 * left:T - 32 * E] = tok[S + 32 * n:T]
                v[s] = want.reshape(-1)
            elif name.endswith("ring"):
                v[s] = np.roll(row.reshape(-1, 256), -32 * E, 0).reshape(-1)
            elif not name.endswith("sink"):
                per = row.reshape(lay.q_cap // 32, -1)
                want = per.copy()
                want[:left] = per[place]
                v[s] = want.reshape(-1)
    return buf, out, source


def records(rng, cfg, lengths, kind):
    shape = (cfg["batch"], cfg["n_kv_heads"], cfg["max_tokens"])
    if kind == "random":
        m = np.exp(3 * rng.standard_normal(shape))
    elif kind == "zero":
        m = np.zeros(shape)
    elif kind == "ties":  # few distinct totals, the same values in other orders among them
        m = np.zeros(shape)
        for j in range(shape[2] // 32 + 1):
            part = m[..., cfg["n_sink"] + 32 * j:cfg["n_sink"] + 32 * j + 32]
            one = np.float32(2.0 ** -20) * np.arange(part.shape[-1]) + (j * 7 % 3)
            part[:] = rng.permutation(one)
    elif kind == "signed":
        m = rng.standard_normal(shape)
    else:  # odd values in places
        m = rng.random(shape)
        m[rng.random(shape) < 0.01] = np.inf
        m[rng.random(shape) < 0.01] = np.nan
        m[rng.random(shape) < 0.01] = -np.inf
        m[rng.random(shape) < 0.1] = 1e-42  # subnormal
    m = m.astype(np.float32)
    for b, T in enumerate(lengths):
        if kind == "random":
            m[b, :, T:] = 0
    return m


def check(B, cfg, lengths, drop, seed, kind="random", in_place=True, stream=None, with_source=True):
    rng = np.random.default_rng(seed)
    layer, _ = fill(B, cfg, lengths, rng)
    # what lies behind the tokens is left as it was: put something there
    mass = records(rng, cfg, lengths, kind)
    buf, want, source = expected(B, layer, cfg, lengths, drop, mass)
    m = torch.from_numpy(mass).cuda()
    other = m if in_place else torch.full_like(m, 5.0)
    src = torch.full(source.shape, -7, dtype=torch.int32, device="cuda") if with_source else None
    ws = B.new_evict_workspace(cfg)
    ws.fill_(0xFF)
    torch.cuda.synchronize()
    left = layer.evict(lengths, drop, m, other, src, ws, stream=stream)
    torch.cuda.synchronize()
    assert left == [t - 32 * e for t, e in zip(lengths, drop)]
    if with_source:
        assert np.array_equal(src.cpu().numpy(), source)
    got = other.cpu().numpy()
    if not in_place:
        for b, T in enumerate(lengths):
            want[b, :, T:] = 5.0
        assert np.array_equal(m.cpu().numpy().view(np.int32), mass.view(np.int32)), "the input record changed"
    assert np.array_equal(got.view(np.int32), want.view(np.int32))
    have = layer.buf.cpu().numpy()
    if not np.array_equal(have, buf):
        at = np.flatnonzero(have != buf)
        where = [n for n in B.REGIONS if getattr(layer.layout, n).offset <= at[0] < getattr(layer.layout, n).offset + getattr(layer.layout, n).bytes]
        raise AssertionError(f"{len(at)} bytes differ, first in {where}")
    return layer, left


LENGTHS = [0, 3, 36, 68, 100, 357, 1000]
DROP = [0, 0, 0, 1, 1, 7, 13]


@pytest.mark.parametrize("form", EVICT)
@pytest.mark.parametrize("in_place", [True, False])
def test_forms(B, form, in_place):
    check(B, config(form, 7, 4, 2, 1024), LENGTHS, DROP, 1, in_place=in_place)


@pytest.mark.parametrize("kind", ["zero", "ties", "signed", "odd"])
@pytest.mark.parametrize("form", ["kv4", "fp16"])
def test_records(B, form, kind):
    check(B, config(form, 3, 3, 3, 2048), [2048, 1500, 357], [20, 1, 9], 2, kind=kind)


@pytest.mark.parametrize("form", ["k8v4", "nuq", "fp16"])
@pytest.mark.parametrize("sink,recent", [(0, 0), (1, 17), (4, 100), (0, 200)])
def test_windows(B, form, sink, recent):
    """Sinks and windows of odd sizes; none, some, nearly all and all groups."""
    cfg = config(form, 5, 2, 1, 900, n_sink=sink, n_recent=recent)
    lengths = [900, 640, 389, 333, 271]
    n = [groups_of(cfg, t) for t in lengths]
    check(B, cfg, lengths, [0, 1, n[2] // 2, n[3] - 1, n[4]], 3)


def test_more_groups_than_threads(B):
    check(B, config("kv2", 1, 1, 1, 70000, n_recent=32), [69990], [700], 4)


def test_nothing_leaves(B):
    check(B, config("kv4", 2, 4, 2, 300), [300, 40], [0, 0], 5, in_place=False)
    check(B, config("kv4", 2, 4, 2, 30), [30, 0], [0, 0], 5, in_place=False)


def test_other_stream_and_no_source(B):
    check(B, config("kv4", 2, 4, 2, 600), [600, 400], [5, 3], 6, stream=torch.cuda.Stream(), with_source=False)


def test_many_rows(B):
    lengths = [(53 * b) % 500 for b in range(90)]
    cfg = config("k4v2", 90, 2, 2, 512)
    check(B, cfg, lengths, [groups_of(cfg, t) // 3 for t in lengths], 7)


def test_captured_and_replayed(B):
    rng = np.random.default_rng(8)
    cfg = config("kv4", 2, 4, 2, 1000)
    a, _ = fill(B, cfg, [1000, 700], rng)
    start = a.buf.clone()
    mass = torch.from_numpy(records(rng, cfg, [1000, 700], "random")).cuda()
    out, ws = torch.zeros_like(mass), B.new_evict_workspace(cfg)
    a.evict([1000, 700], [9, 4], mass, out, None, ws)
    torch.cuda.synchronize()
    want, record = a.buf.clone(), out.clone()
    a.buf.copy_(start)
    out.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.evict([1000, 700], [9, 4], mass, out, None, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.buf, want) and torch.equal(out, record)


def test_the_cache_goes_on(B):
    """After an eviction the window rule's counts hold and the cache takes appends and decodes."""
    rng = np.random.default_rng(9)
    cfg = config("kv4", 2, 4, 2, 700)
    layer, left = check(B, cfg, [700, 411], [6, 3], 10)
    for T, t, e in zip(left, [700, 411], [6, 3]):
        assert counts(cfg, T)[1] == counts(cfg, t)[1] - 32 * e and counts(cfg, T)[2] == counts(cfg, t)[2]
