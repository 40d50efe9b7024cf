"""Tokens that are taken back (drafted ones that were not accepted): the plan against a
request-by-request model, blocks that come back, the cache after it."""
import random

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_kv_cache_07_gb300 import blocks  # noqa: E402
from tests._block_testutil import BLOCK, D, Plan, attention, half_step, values  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


def dev(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Back(Plan):
    """kvq_block_plan_back, request by request."""

    def step_back(self, n_new, n_back):
        new = list(n_new)
        for b, (n, back) in enumerate(zip(n_new, n_back)):
            l = self.lens[b]
            if n < 0:
                left = 0
            elif 0 <= back <= l:
                left = l - back
            else:  # served nothing
                new[b] = BLOCK * self.M + 1
                continue
            for j in range(-(-left // BLOCK), -(-l // BLOCK)):
                self.stack[self.free] = int(self.table[b, j])
                self.free += 1
            self.lens[b] = left
        return self.step(new)


def pair(batch, n_tokens, n_blocks, max_blocks):
    cfg = dict(batch=batch, n_tokens=n_tokens, n_q_heads=1, n_kv_heads=1, head_dim=128, n_blocks=n_blocks, max_blocks=max_blocks)
    return Back(batch, n_tokens, n_blocks, max_blocks), blocks.Tables(cfg)


def held(model):
    return [int(model.table[b, j]) for b in range(model.B) for j in range(-(-model.lens[b] // BLOCK))]


# one CTA's slots and several CTAs', pools that run out
@pytest.mark.parametrize("batch,n_tokens,n_blocks,max_blocks", [
    (1, 1, 1, 1), (1, 70, 3, 3), (3, 64, 7, 4), (16, 90, 40, 9), (33, 1500, 60, 8), (64, 640, 64, 64), (200, 5000, 300, 20),
    (1024, 9000, 700, 12)])
def test_steps(batch, n_tokens, n_blocks, max_blocks):
    r = random.Random(batch + n_tokens)
    model, t = pair(batch, n_tokens, n_blocks, max_blocks)
    for _ in range(14):
        few = max(1, n_tokens // batch)
        new = [r.choice([0, 1, 5, 5, -1, r.randrange(0, 2 * few + 2), r.randrange(0, BLOCK * max_blocks + 2)]) for _ in range(batch)]
        back = [r.choice([0, 0, 1, 4, l, r.randint(0, l), r.randint(0, l), l + 1, -1]) for l in model.lens]
        t.plan(dev(new), n_back=dev(back))
        model.step_back(new, back).same(t)
        ids = held(model) + model.stack[:model.free]
        assert sorted(ids) == list(range(n_blocks))  # nothing is lost, nothing held twice


def test_a_request_gives_and_takes_in_one_step():
    """Blocks behind the new length come back while the same table entries get new ones."""
    model, t = pair(2, 400, 8, 6)
    for new, back in (([150, 40], [0, 0]), ([100, 0], [120, 0]), ([0, 90], [128, 33]), ([1, -1], [2, 5]), ([180, 3], [1, 0]), ([0, 0], [181, 0])):
        t.plan(dev(new), n_back=dev(back))
        model.step_back(new, back).same(t)


def test_zeros_are_a_plan():
    """No tokens back: what the plan without them gives."""
    r = random.Random(5)
    (model, t), (_, u) = pair(9, 200, 40, 8), pair(9, 200, 40, 8)
    for _ in range(8):
        new = dev([r.choice([1, 1, 40, -1, 0]) for _ in range(9)])
        t.plan(new, n_back=torch.zeros_like(new))
        u.plan(new)
        for name in ("block_table", "free_list", "free_count", "lens", "start", "unit0", "token_row", "position", "slot"):
            assert torch.equal(getattr(t, name), getattr(u, name)), name


def test_lengths_apart_and_captured():
    """Lengths of their own make the call repeatable; a captured one takes the step's numbers."""
    model, t = pair(3, 100, 12, 4)
    model.step_back([50, 33, 10], [0, 0, 0])
    t.plan(dev([50, 33, 10]))
    lens, count, new, back = t.lens.clone(), t.free_count.clone(), dev([5, 5, 5]), dev([20, 1, 0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        t.plan(new, lens=lens, free_count=count, n_back=back)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            t.plan(new, n_back=back)
    torch.cuda.current_stream().wait_stream(side)
    model.step_back([5, 5, 5], [20, 1, 0]).same(t)
    for n, b in (([5, 5, 5], [4, 2, 0]), ([5, -1, 33], [40, 9, 5]), ([5, 70, 1], [0, 0, 43])):
        new.copy_(dev(n))
        back.copy_(dev(b))
        graph.replay()
        model.step_back(n, b).same(t)


def test_refused_tensors():
    _, t = pair(4, 50, 10, 3)
    new = dev([1, 1, 1, 1])
    for bad in (new.long(), dev([0] * 5), new.cpu(), dev([0] * 8)[::2], [0, 0, 0, 0]):
        with pytest.raises(ValueError):
            t.plan(new, n_back=bad)


def test_drafted_tokens():
    """Chains of five drafted tokens of which few are accepted: the pool keeps its blocks,
    the cache holds the accepted tokens, attention is of them and the new ones alone."""
    B, N, HQ, HKV, NB, MB = 3, 15, 4, 2, 30, 7
    cfg = dict(batch=B, n_tokens=N, n_q_heads=HQ, n_kv_heads=HKV, head_dim=128, n_blocks=NB, max_blocks=MB)
    rng, r = np.random.default_rng(0), random.Random(1)
    model, t = Back(B, N, NB, MB), blocks.Tables(cfg)
    layer, ws = blocks.Layer(cfg), blocks.new_workspace(cfg)
    rows, back = [[] for _ in range(B)], [0] * B
    for step in range(40):
        new = [r.choice([5, 5, 5, 0]) for _ in range(B)]
        x = rng.standard_normal((N, HQ + 2 * HKV, D)).astype(np.float16)
        g = torch.from_numpy(x).cuda()
        q = g[:, :HQ].contiguous()
        out, lse = torch.full_like(q, 7.0), torch.full((N, HQ), 7.0, device="cuda")
        t.plan(dev(new), n_back=dev(back))
        model.step_back(new, back).same(t)
        layer.append(t, g[:, HQ:HQ + HKV], g[:, HQ + HKV:])
        layer.attn(t, q, out, lse, ws)
        assert model.free + len(held(model)) == NB
        kv = values(layer.codes.cpu().numpy(), layer.scales.cpu().numpy())
        o, s, scales = out.cpu().numpy().astype(float), lse.cpu().numpy(), layer.scales.cpu().numpy()
        for b in range(B):
            a, e, L = model.start[b], model.start[b + 1], model.lens[b]
            rows[b] = rows[b][:len(rows[b]) - back[b]] + [x[i, HQ:].astype(float).reshape(2, HKV, D).transpose(1, 0, 2) for i in range(a, e)]
            assert len(rows[b]) == L
            if L:
                ids = model.table[b, :-(-L // BLOCK)]
                got = kv[ids].transpose(0, 3, 1, 2, 4).reshape(-1, HKV, 2, D)[:L]
                want = np.array(rows[b])
                unit = (2.0 ** (scales[ids].astype(float) - 127)).repeat(BLOCK, 0)[:L, ..., None]
                # half a step of the code, and half of the smallest one where the block's scale grew
                # (no more than once: normal values have maxima of 3 to 6 in four tokens or more)
                assert (np.abs(got - want) <= half_step(np.abs(want) / unit) * unit + 2 * 2.0**-10 * unit).all()
            if a < e:
                wo, wl = attention(x[a:e, :HQ], kv, model.table[b], L, e - a, HQ, HKV)
                vmax = np.abs(kv[model.table[b, :-(-L // BLOCK)], :, 1]).max()
                assert (np.abs(o[a:e] - wo) <= 2.0**-10 * vmax + 2.0**-16 * vmax).all() and (np.abs(s[a:e] - wl) <= 2.0**-15).all()
            back[b] = r.randint(0, e - a) if a < e else 0
