"""The block cache without a GPU: sizes, refusals of the C ABI before any launch,
the schedule's helpers' agreement with the formats of the tests."""
import ctypes as C

import numpy as np
import pytest

from bit_kv_cache_07_gb300 import binding, blocks
from tests._block_testutil import E4M3, exponent, half_step, unswizzled


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


def config(**kw):
    c = dict(batch=4, n_tokens=8, n_q_heads=8, n_kv_heads=2, head_dim=128, n_blocks=33, max_blocks=5, rope_theta=10000.0,
             norm_eps=1e-6)
    c.update(kw)
    return blocks.make_config(c)


def test_layout():
    L = blocks.layout(config())
    assert L.codes_bytes == 33 * 2 * 2 * 32 * 128
    assert L.scales_bytes == (33 * 2 * 2 + 15) // 16 * 16 and L.workspace_bytes > 0


@pytest.mark.parametrize("field,value,status", [
    ("batch", 0, -1), ("batch", 1025, -2), ("n_tokens", 0, -1), ("n_tokens", (1 << 20) + 1, -2), ("n_q_heads", 7, -1),
    ("n_q_heads", 0, -1), ("n_q_heads", 4096, -2), ("n_kv_heads", 0, -1), ("head_dim", 64, -2), ("n_blocks", 0, -1), ("n_blocks", (1 << 26) + 1, -2),
    ("max_blocks", 0, -1), ("max_blocks", (1 << 25) + 1, -2), ("window", -1, -1), ("n_first", -1, -1),
    ("softmax_scale", -1.0, -1), ("softmax_scale", float("nan"), -1), ("rope_theta", float("inf"), -1),
    ("rope_theta", -1.0, -1), ("norm_eps", float("nan"), -1), ("norm_eps", -1.0, -1)])
def test_config_refusals(field, value, status):
    with pytest.raises(binding.KvqError) as e:
        blocks.layout(config(**{field: value}))
    assert e.value.status == status


def test_too_many_rows():
    with pytest.raises(binding.KvqError) as e:
        blocks.layout(config(n_tokens=1 << 20, n_q_heads=2048, n_kv_heads=16))
    assert e.value.status == -2


def test_unknown_names():
    with pytest.raises(ValueError):
        blocks.make_config(dict(batch=1, heads=3))


A = 1 << 20  # an address that is never read: every call below is refused before a launch


def tables(**kw):
    t = {n: A for n in binding.BLOCK_TABLES}
    t.update(kw)
    return binding.kvq_block_tables(*[t[n] for n in binding.BLOCK_TABLES])


def test_plan_refusals():
    L, c = binding.lib(), config()
    ok = [C.byref(c), C.byref(tables()), A, A, A, None]
    for i, bad in ((0, None), (1, None), (2, None), (3, None), (4, None), (2, A + 2), (3, A + 1), (4, A + 2)):
        args = list(ok)
        args[i] = bad
        assert L.kvq_block_plan(*args) == -1, (i, bad)
    for n in binding.BLOCK_TABLES:
        for bad in (None, A + 2):
            assert L.kvq_block_plan(C.byref(c), C.byref(tables(**{n: bad})), A, A, A, None) == -1, n
    assert L.kvq_block_plan(C.byref(config(batch=2000)), C.byref(tables()), A, A, A, None) == -2


def test_append_refusals():
    L, c = binding.lib(), config()
    K, V, Q, O = A, 2 * A, 3 * A, 4 * A  # far apart
    kv, q = 2 * 128, 8 * 128
    names = ["cfg", "tables", "codes", "scales", "k", "k_stride", "v", "v_stride", "q", "q_stride", "q_out", "q_weight", "k_weight", "stream"]
    ok = dict(cfg=C.byref(c), tables=C.byref(tables()), codes=A, scales=A, k=K, k_stride=kv, v=V, v_stride=kv, q=Q, q_stride=q, q_out=O,
              q_weight=A, k_weight=A, stream=None)

    def call(**kw):
        a = dict(ok, **kw)
        return L.kvq_block_append(*[a[n] for n in names])
    for name in ("cfg", "tables", "codes", "scales", "k", "v", "q", "q_out"):
        assert call(**{name: None}) == -1, name
    for name in ("codes", "scales", "k", "v", "q", "q_out", "q_weight", "k_weight"):
        assert call(**{name: ok[name] + 8}) == -1, name
    for name, row in (("k_stride", kv), ("v_stride", kv), ("q_stride", q)):
        for bad in (row - 8, row + 4, 0, -row, 1 << 41):
            assert call(**{name: bad}) == -1, (name, bad)
    assert call(q=None, q_out=None) == -1          # a weight without queries
    assert call(q_out=Q, q_stride=q + 128) == -1   # in place, but not dense
    assert call(q_out=Q + 256) == -1               # overlaps q
    assert call(q_out=K + 1024) == -1              # overlaps k
    assert call(q_out=V - 2 * q * 7) == -1         # overlaps v
    # one projection's rows: q_out inside them is refused
    assert call(q=A, q_stride=q + 2 * kv, k=A + 2 * q, k_stride=q + 2 * kv, v=A + 2 * (q + kv), v_stride=q + 2 * kv, q_out=A) == -1


def test_attn_refusals():
    L, c = binding.lib(), config()
    ws = blocks.layout(c).workspace_bytes
    names = ["cfg", "tables", "codes", "scales", "q", "out", "lse", "workspace", "ws_bytes", "stream"]
    ok = dict(cfg=C.byref(c), tables=C.byref(tables()), codes=A, scales=A, q=2 * A, out=3 * A, lse=A, workspace=A, ws_bytes=ws, stream=None)

    def call(**kw):
        a = dict(ok, **kw)
        return L.kvq_block_attn(*[a[n] for n in names])
    for name in ("cfg", "tables", "codes", "scales", "q", "out"):
        assert call(**{name: None}) == -1, name
    for name in ("codes", "scales", "q", "out"):
        assert call(**{name: ok[name] + 8}) == -1, name
    assert call(lse=A + 2) == -1
    assert call(out=2 * A) == -1 and call(out=2 * A + 1024) == -1  # q is read while out is written
    assert call(workspace=None) == -4 and call(workspace=A + 8) == -4 and call(ws_bytes=ws - 1) == -4


def test_formats_of_the_tests():
    """The tests' own e4m3: 448 the largest, steps as half_step says, rows told apart."""
    assert np.nanmax(E4M3) == 448.0 and E4M3[1] == 2.0**-9 and E4M3[0x38] == 1.0 and np.isnan(E4M3[0x7F]) and np.isnan(E4M3[0xFF])
    v = E4M3[:127]
    gaps = np.diff(v)
    assert np.allclose(gaps / 2, half_step(v[:-1])) and (gaps > 0).all()
    torch = pytest.importorskip("torch")
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref, E4M3, equal_nan=True)
    assert [exponent(x) for x in (0, 448, 448.0001, 896, 3.5, 3.51, 1e-20, 1e30)] == [-40, 0, 1, 1, -7, -6, -40, 40]
    b = np.zeros((32, 128), np.uint8)
    b[5, (3 ^ 5) * 16 + 7] = 9  # token 5, chunk 3
    u = unswizzled(b)
    assert u[5, 3 * 16 + 7] == 9 and u.sum() == 9
