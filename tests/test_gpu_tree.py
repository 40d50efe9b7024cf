"""kvq_tree_attn on the GPU against attention in 64 bits: every cache form,
row lengths from an empty cache over window boundaries to several tiles,
node counts from one to 256 with odd ones, masks of trees, of nothing and of
scattered bits, and values behind a mask that are not finite.

Tolerances.  The kernel rounds each value (2^-11 of it at most, half a step of
fp16) and each attention weight (2^-11, plus 2^-25 absolute for weights in
fp16's subnormal range relative to a maximum of 1), its logits carry 2^-20 of
sum |q k| scale, and the result rounds to fp16 once: elementwise
  |err| <= 2^-11 |out| + (2 * 2^-11 + 2 E) sum_t w_t |v_t| + 2^-24,
E the logit error (weights change by e^E - 1, numerator and denominator).  The
stored values of a Hadamard-rotated cache carry their errors through the
rotation: the 2-norm of the same bound takes the sum's place."""
import numpy as np
import pytest
import torch

from _spec_testutil import FORMS, attention, cached, config, fill, random_kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


def tree_masks(B, rng, batch, n, counts):
    parents = np.stack([[int(rng.integers(max(-1, i - 6), i)) if i else -1 for i in range(n)] for _ in range(batch)])
    return B.tree_mask(parents)


def bits(words, n):
    w = words.numpy().astype("<i4").view(np.uint8)
    return np.unpackbits(w.reshape(*words.shape[:-1], -1), axis=-1, bitorder="little")[..., :n].astype(bool)


def check(B, cfg, lengths, n, nodes=None, seed=0, mask="tree", poison=False):
    rng = np.random.default_rng(seed)
    layer, stores = fill(B, cfg, lengths, rng)
    batch, hq, hkv = cfg["batch"], cfg["n_q_heads"], cfg["n_kv_heads"]
    g = hq // hkv
    q = rng.standard_normal((batch, hq, n, 128)).astype(np.float16)
    kd, vd = random_kv(rng, (batch, hkv, n, 128))
    count = [n] * batch if nodes is None else nodes
    if mask == "tree":
        words = tree_masks(B, rng, batch, n, count)
    elif mask == "scattered":  # any pattern, rows that see no drafted token among them, bits past the nodes set
        words = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (batch, n, (n + 31) // 32)).astype(np.int32))
        words[:, ::3] = 0
    else:
        words = None
    sees = np.zeros((batch, n, n), bool) if words is None else bits(words, n)
    if poison:  # the last node of every row is seen by itself alone, the one before by nobody
        for b in range(batch):
            sees[b, :, n - 1], sees[b, :, n - 2] = False, False
            sees[b, n - 1, n - 1] = True
        packed = np.packbits(np.pad(sees, ((0, 0), (0, 0), (0, -n % 32))).reshape(batch, n, -1, 32), axis=-1, bitorder="little")
        words = torch.from_numpy(np.ascontiguousarray(packed).view("<i4")[..., 0].copy())
        kd[:, :, n - 2], vd[:, :, n - 2] = np.nan, np.inf
        vd[:, :, n - 1, :5] = np.nan
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    ws = B.new_tree_workspace(cfg, n)
    ws.fill_(0xFF)  # scratch contents mean nothing
    layer.tree_attn(lengths, t(q), t(kd), t(vd), None if words is None else words.cuda(), out, lse, ws, nodes)
    first = (out.clone(), lse.clone())
    layer.tree_attn(lengths, t(q), t(kd), t(vd), None if words is None else words.cuda(), out, lse, ws, nodes)
    torch.cuda.synchronize()
    assert torch.equal(first[0].view(torch.int16), out.view(torch.int16)) and torch.equal(first[1].view(torch.int32), lse.view(torch.int32))
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    scale = cfg["softmax_scale"] or 1 / np.sqrt(128.0)
    for s, store in enumerate(stores):
        b, h = divmod(s, hkv)
        m, T = count[b], lengths[b]
        k, v, stored, quant = cached(cfg, store, T)
        k = np.concatenate([k, kd[b, h, :m].astype(np.float64)])
        dv = vd[b, h, :m].astype(np.float64)
        v, stored, quant = np.concatenate([v, dv]), np.concatenate([stored, dv]), np.concatenate([quant, np.zeros(m, bool)])
        for j in range(g):
            head = h * g + j
            assert (out[b, head, m:] == 7.0).all() and (lse[b, head, m:] == 7.0).all(), "slots past the nodes changed"
            for i in range(m):
                see = np.concatenate([np.ones(T, bool), sees[b, i, :m]])
                qi = q[b, head, i:i + 1].astype(np.float64)
                ref, rl, spread, rotated, direct = attention(qi, k[see], v[see], stored[see], quant[see], scale)
                got = out[b, head, i]
                where = (b, head, i, T)
                if not see.any():
                    assert (got == 0).all() and lse[b, head, i] == -np.inf, where
                    continue
                E = 2.0 ** -20 * scale * (np.abs(qi) @ np.abs(k[see]).T).max()
                weigh = rotated if cfg["v_hadamard"] else direct
                bound = 2.0 ** -11 * np.abs(ref) + (2.0 ** -10 + 2 * E) * (spread + weigh[:, None] if cfg["v_hadamard"] else spread + weigh) + 2.0 ** -24
                bad = ~np.isfinite(ref[0])
                assert (np.isnan(got) | np.isinf(got))[bad].all(), where
                assert (np.abs(got - ref[0]) <= bound[0])[~bad].all(), (where, np.max((np.abs(got - ref[0]) / bound[0])[~bad]))
                # logits and their sum: E, and fp32 roundings of the exponent and the logarithm
                assert abs(lse[b, head, i] - rl[0]) <= E + 2.0 ** -20 * max(1.0, abs(rl[0])), (where, lse[b, head, i], rl[0])


LENGTHS = [0, 1, 35, 36, 67, 68, 300, 997]


@pytest.mark.parametrize("n", [5, 9])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_forms(B, form, n):
    """10 and 18 rows per KV head: the two kernels."""
    check(B, config(form, 8, 4, 2, 1024), LENGTHS, n, seed=1)


@pytest.mark.parametrize("g,n", [(1, 1), (1, 16), (1, 17), (3, 11), (4, 16), (7, 9), (8, 16), (8, 33), (2, 65), (1, 130), (8, 256)])
def test_rows(B, g, n):
    """Rows per KV head around the row blocks (16, 32, 64, 128 and several)."""
    check(B, config("kv4", 2, 2 * g, 2, 700), [517, 40], n, seed=2)


@pytest.mark.parametrize("form", ["kv8", "k4v2_hadamard", "fp16", "nuq_rope"])
@pytest.mark.parametrize("n", [16, 63])
def test_node_counts(B, form, n):
    """Rows that use part of their slots, or none."""
    check(B, config(form, 5, 8, 2, 512, n_sink=0, n_recent=0), [0, 333, 96, 500, 31], n, nodes=[n, 0, 1, n - 3, 7], seed=3)


@pytest.mark.parametrize("form", ["kv4", "fp16", "k4v2_hadamard"])
def test_scattered_masks(B, form):
    check(B, config(form, 3, 4, 1, 400), [0, 200, 399], 45, nodes=[45, 38, 3], seed=4, mask="scattered")


@pytest.mark.parametrize("form", ["kv4", "fp16", "nuq"])
def test_no_drafted_tokens(B, form):
    check(B, config(form, 3, 4, 2, 400), [0, 200, 399], 6, seed=5, mask=None)


@pytest.mark.parametrize("form", ["kv4", "fp16"])
@pytest.mark.parametrize("n", [7, 40])
def test_not_finite_behind_the_mask(B, form, n):
    check(B, config(form, 3, 4, 2, 400), [0, 200, 399], n, seed=6, poison=True)


def test_many_rows_of_a_batch(B):
    check(B, config("k8v4", 70, 2, 2, 300, n_recent=17), [(37 * b) % 300 for b in range(70)], 3, seed=7)


def test_head_subset(B):
    """A cache that holds three of a layer's five KV heads, in another order."""
    rng = np.random.default_rng(8)
    heads, g, n, T = [3, 0, 4], 2, 7, 260
    cfg = config("kv4", 2, 6, 3, 300, kv_heads_total=5, kv_head_index=heads)
    K, V = random_kv(rng, (2, 5, T, 128))
    q = rng.standard_normal((2, 10, n, 128)).astype(np.float16)
    kd, vd = random_kv(rng, (2, 5, n, 128))
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    words = tree_masks(B, rng, 2, n, [n, n])
    plain = config("kv4", 2, 10, 5, 300)
    whole, part = B.Layer(plain), B.Layer(cfg)
    for layer in (whole, part):
        layer.append(0, t(K), t(V))
    outs = []
    for layer, c in ((whole, plain), (part, cfg)):
        out = torch.zeros(q.shape, dtype=torch.float16, device="cuda")
        lse = torch.zeros(q.shape[:3], device="cuda")
        layer.tree_attn([T, T - 9], t(q), t(kd), t(vd), words.cuda(), out, lse, B.new_tree_workspace(c, n))
        outs.append((out.cpu(), lse.cpu()))
    for h in range(5):
        rows = slice(h * g, (h + 1) * g)
        if h in heads:  # the same tiles, cut at other places
            assert torch.allclose(outs[0][0][:, rows].float(), outs[1][0][:, rows].float(), rtol=2 ** -9, atol=2 ** -9)
            assert torch.allclose(outs[0][1][:, rows], outs[1][1][:, rows], rtol=1e-5)
        else:
            assert not outs[1][0][:, rows].any() and not outs[1][1][:, rows].any()


def test_captured_replayed_and_other_stream(B):
    rng = np.random.default_rng(9)
    cfg = config("k8v4", 2, 8, 2, 600)
    layer, _ = fill(B, cfg, [600, 411], rng)
    n = 12
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    q = t(rng.standard_normal((2, 8, n, 128)).astype(np.float16))
    kd, vd = (t(x) for x in random_kv(rng, (2, 2, n, 128)))
    words = tree_masks(B, rng, 2, n, [n, n]).cuda()
    out, lse, ws = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda"), B.new_tree_workspace(cfg, n)
    call = lambda **kw: layer.tree_attn([600, 411], q, kd, vd, words, out, lse, ws, **kw)  # noqa: E731
    call()
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    call(stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    q.mul_(0.5)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    call()
    torch.cuda.synchronize()
    assert torch.equal(out, replayed) and not torch.equal(out, want)


def test_agrees_with_the_decode(B):
    """One node that sees itself alone, appended instead: the same attention."""
    rng = np.random.default_rng(10)
    cfg = config("kv4", 2, 8, 2, 600)
    layer, _ = fill(B, cfg, [500, 77], rng)
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    q = t(rng.standard_normal((2, 8, 1, 128)).astype(np.float16))
    kd, vd = (t(x) for x in random_kv(rng, (2, 2, 1, 128)))
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    layer.tree_attn([500, 77], q, kd, vd, B.tree_mask([[-1], [-1]]).cuda(), out, lse, B.new_tree_workspace(cfg, 1))
    layer.append_ragged([500, 77], [1, 1], kd, vd)
    o2, l2 = torch.zeros_like(q[:, :, 0]), torch.zeros(2, 8, device="cuda")
    layer.decode_ragged([501, 78], q[:, :, 0].contiguous(), o2, l2, B.new_workspace(cfg))
    torch.cuda.synchronize()
    assert torch.allclose(lse[:, :, 0], l2, rtol=1e-5, atol=1e-5)
    assert torch.allclose(out[:, :, 0].float(), o2.float(), rtol=4e-3, atol=4e-3)
