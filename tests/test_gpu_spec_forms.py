"""Forms of a cache that the other tests of tree attention and the record leave
out: uniform codes whose scales pass fp16's range within the operands, and
non-uniform codes without outliers.

Tolerances of the wide scales.  A key is min + 2^(b-1) s + c' s, parts below
131,008 in size each; logits are sums of 128 products per part in fp32, and c' s
enters in two fp16 parts.  Past 65,504 the second part holds what exceeds it:
up to 288 (8 bits), 4,400 (4) or 21,856 (2), off by half a step of fp16 there,
1/8, 2 or 8.  So E = scale sum |q| (2^-20 * 3 * 131,008 + that).  A value rounds
to fp16, 2^-11, and one that the scale's own rounding (2^-11 of up to 131,008)
has put past fp16's range saturates, off by 64 at most; the output's sums as in
test_gpu_spec_range."""
import numpy as np
import pytest
import torch

from _spec_testutil import attention, build_row, cached, config, random_kv
from test_gpu_mass import check as check_mass
from test_gpu_spec_scales import check_mass as check_mass_of
from test_gpu_tree import check as check_tree

pytestmark = pytest.mark.gpu
BEYOND = {8: 0.125, 4: 2.0, 2: 8.0}


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


def wide(rng, shape):
    """Keys and values up to fp16's largest number, of both signs in every
    group of 32 tokens and of 32 channels."""
    x = rng.uniform(-65504.0, 65504.0, shape)
    x[..., ::8, ::4], x[..., 1::8, ::4] = 65504.0, -65504.0
    x[..., 2::8, 1::4], x[..., 2::8, 2::4] = 65504.0, -65504.0
    return x.astype(np.float16)


def errors(cfg, q):
    return (np.abs(q).sum(-1) / np.sqrt(128.0)) * (2.0 ** -20 * 3 * 131008.0 + BEYOND[cfg["k_bits"]])


@pytest.mark.parametrize("form", ["kv8", "k8v4", "kv4", "k4v2", "kv2", "k2v8", "kv4_g32"])
@pytest.mark.parametrize("n", [5, 9])
def test_wide_scales(B, form, n):
    rng = np.random.default_rng(90)
    lengths, hkv, g = [300, 133], 2, 2
    cfg = config(form, 2, hkv * g, hkv, 300)
    K, V = wide(rng, (2, hkv, 300, 128)), wide(rng, (2, hkv, 300, 128))
    q = (1e-4 * rng.standard_normal((2, hkv * g, n, 128))).astype(np.float16)
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    layer = B.Layer(cfg)
    layer.append_ragged([0, 0], lengths, t(K), t(V))
    out, lse = torch.zeros(q.shape, dtype=torch.float16, device="cuda"), torch.zeros(q.shape[:3], device="cuda")
    layer.tree_attn(lengths, t(q), None, None, None, out, lse, B.new_tree_workspace(cfg, n))
    got, gl = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    past = 0
    for b, T in enumerate(lengths):
        for h, store in enumerate(build_row(cfg, K[b], V[b], T)):
            k, v, stored, quant = cached(cfg, store, T)
            past = max(past, np.abs(k[quant]).max(), np.abs(v[quant]).max())
            for head in range(h * g, (h + 1) * g):
                qs = q[b, head].astype(np.float64)
                ref, rl, a, _, w = attention(qs, k, v, stored, quant, 1 / np.sqrt(128.0))
                E = errors(cfg, qs)
                weights = 2.0 ** -20 + (T + 30) * 2.0 ** -26 + 2.0 ** -11 + 2 * E[:, None]
                bound = 2.0 ** -11 * np.abs(ref) + 64.0 + weights * (a + w) + 2.0 ** -31 * np.abs(v).sum(0)
                assert (np.abs(got[b, head] - ref) <= bound).all(), (b, head, np.max(np.abs(got[b, head] - ref) / bound))
                assert (np.abs(gl[b, head] - rl) <= E + 2.0 ** -20 * np.maximum(1.0, np.abs(rl))).all()
    assert past > 65504.0  # values and keys that the scale has put past the range are among them


@pytest.mark.parametrize("form", ["kv8", "kv4", "kv2"])
@pytest.mark.parametrize("g,n", [(1, 1), (2, 4), (3, 3), (5, 13)])
def test_record_of_wide_scales(B, form, g, n):
    rng = np.random.default_rng(91)
    lengths, hkv = [300, 133], 2
    cfg = config(form, 2, hkv * g, hkv, 300)
    K, V = wide(rng, (2, hkv, 300, 128)), wide(rng, (2, hkv, 300, 128))
    q = (1e-4 * rng.standard_normal((2, hkv * g, n, 128))).astype(np.float16)
    check_mass_of(B, cfg, lengths, K, V, q, more=errors(cfg, q.astype(np.float64)).max())


@pytest.mark.parametrize("form", ["nuq", "nuq_hadamard", "nuq_rope"])
@pytest.mark.parametrize("n", [5, 9])
def test_non_uniform_codes_without_outliers(B, form, n):
    cfg = config(form, 3, 4, 2, 700, outliers_per_vector=0)
    check_tree(B, cfg, [670, 0, 131], n, seed=92)
    check_mass(B, cfg, [670, 0, 131], n, 93)
