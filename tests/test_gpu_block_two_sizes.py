"""Two configurations over one cache, as the README shows: steps of single tokens with a slot
for each request, and steps with room for prompts.  Both share the requests' arrays and the
layer's memory; each has its own offsets and slot maps."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_kv_cache_07_gb300 import blocks  # noqa: E402
from tests._block_testutil import D, EPS, Plan, attention, values  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


B, HQ, HKV, NB, MB = 5, 8, 2, 60, 12
STEPS = [[40, 0, 3, 200, 0], [1, 1, 1, 1, 0], [1, 0, 1, 1, 1], [1, -1, 300, 1, 33], [1, 1, 1, 1, 1], [1, 1, -1, 1, 1], [1, 90, 1, -1, 1], [1, 1, 1, 1, 1]]


def test_prompts_and_single_tokens():
    cfg = dict(batch=B, n_tokens=B, n_q_heads=HQ, n_kv_heads=HKV, head_dim=128, n_blocks=NB, max_blocks=MB, rope_theta=10000.0, norm_eps=EPS)
    wide = dict(cfg, n_tokens=400)
    tables = blocks.Tables(cfg)
    layer, ws = blocks.Layer(cfg), blocks.new_workspace(cfg)
    shared = {n: getattr(tables, n) for n in ("block_table", "free_list", "free_count", "lens")}
    kinds = {B: (tables, layer), 400: (blocks.Tables(wide, **shared), blocks.Layer(wide, codes=layer.codes, scales=layer.scales))}
    models = {n: Plan(B, n, NB, MB) for n in kinds}
    models[400].lens, models[400].table, models[400].stack = models[B].lens, models[B].table, models[B].stack
    rng, free = np.random.default_rng(2), NB
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(D)).astype(np.float16)).cuda()
    for new in STEPS:
        n = B if max(new) <= 1 else 400
        (t, one), model = kinds[n], models[n]
        x = torch.from_numpy(rng.standard_normal((n, HQ + 2 * HKV, D)).astype(np.float16)).cuda()
        q, out, lse = torch.zeros((n, HQ, D), dtype=torch.float16, device="cuda"), torch.zeros((n, HQ, D), dtype=torch.float16, device="cuda"), torch.zeros((n, HQ), device="cuda")
        t.plan(torch.tensor(new, dtype=torch.int32, device="cuda"))
        one.append(t, x[:, HQ:HQ + HKV], x[:, HQ + HKV:], x[:, :HQ], q, w, w)
        one.attn(t, q, out, lse, ws)
        model.free = free
        model.step(new).same(t)
        free = model.free
        kv = values(layer.codes.cpu().numpy(), layer.scales.cpu().numpy())
        gq, go, gl = q.cpu().numpy(), out.cpu().numpy().astype(float), lse.cpu().numpy()
        for b in range(B):
            a, e, L = model.start[b], model.start[b + 1], model.lens[b]
            if a == e:
                continue
            o, s = attention(gq[a:e], kv, model.table[b], L, e - a, HQ, HKV)
            vmax = np.abs(kv[model.table[b, :-(-L // 32)], :, 1]).max()
            assert (np.abs(go[a:e] - o) <= 2.0**-10 * vmax + 2.0**-16 * vmax).all() and (np.abs(gl[a:e] - s) <= 2.0**-15).all()
