"""The block cache as a serving loop uses it: one captured step, replayed while
requests start, grow, are refused, end and hand their blocks on, over two layers (one
with a sliding window); every step against 64 bits from the bytes that it stored."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_kv_cache_07_gb300 import blocks  # noqa: E402
from tests._block_testutil import D, EPS, Plan, attention, normed_rotated, values  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


B, N, HQ, HKV, NB, MB = 4, 80, 4, 2, 14, 6
BASE = dict(batch=B, n_tokens=N, n_q_heads=HQ, n_kv_heads=HKV, head_dim=128, n_blocks=NB, max_blocks=MB, rope_theta=10000.0, norm_eps=EPS)
STEPS = [[40, 0, 3, 0], [1, 70, 1, 0], [1, 1, 1, 0], [5, 1, 1, 1], [1, -1, 30, 1], [1, 33, 1, 1], [-1, 1, 1, 80], [64, 1, 1, 1], [1, 1, 1, -1],
         [1, 1, 1, 1]]


@pytest.mark.parametrize("captured", [False, True])
def test_loop(captured):
    rng = np.random.default_rng(1)
    cfgs = [dict(BASE), dict(BASE, window=24, n_first=2)]
    t, plan = blocks.Tables(BASE), Plan(B, N, NB, MB)
    layers, ws = [blocks.Layer(c) for c in cfgs], blocks.new_workspace(BASE)
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    x = [torch.zeros((N, HQ + 2 * HKV, D), dtype=torch.float16, device="cuda") for _ in cfgs]
    q = [torch.zeros((N, HQ, D), dtype=torch.float16, device="cuda") for _ in cfgs]
    out, lse = [torch.zeros_like(q[0]) for _ in cfgs], [torch.zeros((N, HQ), device="cuda") for _ in cfgs]
    w = [torch.from_numpy((1 + 0.1 * rng.standard_normal(D)).astype(np.float16)).cuda() for _ in range(2)]

    def step():
        t.plan(new)
        for i, layer in enumerate(layers):
            layer.append(t, x[i][:, HQ:HQ + HKV], x[i][:, HQ + HKV:], x[i][:, :HQ], q[i], w[0], w[1])
            layer.attn(t, q[i], out[i], lse[i], ws)

    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # of no tokens
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step()
        torch.cuda.current_stream().wait_stream(side)
    rows = [[[] for _ in range(B)] for _ in cfgs]  # keys and values that each request should hold
    for n_new in STEPS:
        for i in range(2):
            x[i].copy_(torch.from_numpy(rng.standard_normal(x[i].shape).astype(np.float16)))
        new.copy_(torch.tensor(n_new, dtype=torch.int32))
        plan.step(n_new)
        graph.replay() if captured else step()
        plan.same(t)
        for i, c in enumerate(cfgs):
            kv = values(layers[i].codes.cpu().numpy(), layers[i].scales.cpu().numpy())
            got, gl, gq, gx = out[i].cpu().numpy().astype(float), lse[i].cpu().numpy(), q[i].cpu().numpy(), x[i].cpu().numpy()
            for b in range(B):
                a, e = plan.start[b], plan.start[b + 1]
                if n_new[b] < 0:
                    rows[i][b] = []
                if a == e:
                    continue
                k = normed_rotated(gx[a:e, HQ:HQ + HKV], w[1].cpu().numpy(), plan.pos[a:e], 10000.0)
                rows[i][b] += [np.stack([k[j], gx[a + j, HQ + HKV:].astype(float)], 1) for j in range(e - a)]
                L = plan.lens[b]
                assert len(rows[i][b]) == L
                # what is stored is the rows to an eighth's half, times the re-rounding of small ones
                ids = plan.table[b, :-(-L // 32)]
                held = kv[ids].transpose(0, 3, 1, 2, 4).reshape(-1, HKV, 2, D)[:L]
                want = np.array(rows[i][b])
                top = np.abs(want).max()
                assert (np.abs(held - want) <= 2.0**-4 * np.abs(want) * 1.01 + 2.0**-13 * top).all()
                o, s = attention(gq[a:e], kv, plan.table[b], L, e - a, HQ, HKV, c.get("window", 0), c.get("n_first", 0))
                vmax = np.abs(held[:, :, 1]).max()
                # 2^-11 of the weights, 2^-11 of the result, logits of |q| |k| <= 12 * 12 / sqrt(128) to 2^-20
                assert (np.abs(got[a:e] - o) <= 2.0**-10 * vmax + 2.0**-16 * vmax).all()
                assert (np.abs(gl[a:e] - s) <= 2.0**-15).all()
