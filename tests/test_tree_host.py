"""kvq_tree_attn's refusals and kvq_tree_workspace, without a GPU: every bad
argument is returned before anything is launched."""
import ctypes as C

import numpy as np
import pytest

from _spec_testutil import config


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    return binding


def call(B, cfg, tokens=(10, 20), n=4, nodes=None, **kw):
    arg = dict(layer=1 << 20, q=1 << 21, kd=1 << 22, vd=1 << 23, mask=1 << 24, out=1 << 25, lse=0, ws=1 << 26, ws_bytes=1 << 40)
    arg.update(kw)
    arr = None if tokens is None else (C.c_int32 * len(tokens))(*tokens)
    nd = None if nodes is None else (C.c_int32 * len(nodes))(*nodes)
    c = B.make_config(cfg)
    return B.lib().kvq_tree_attn(C.byref(c), arg["layer"] or None, arr, arg["q"] or None, arg["kd"] or None, arg["vd"] or None,
                                 arg["mask"] or None, n, nd, arg["out"] or None, arg["lse"] or None, arg["ws"] or None,
                                 arg["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(layer=0), -1), (dict(q=0), -1), (dict(out=0), -1), (dict(tokens=None), -1), (dict(kd=0), -1), (dict(vd=0), -1),
    (dict(layer=(1 << 20) + 8), -1), (dict(q=(1 << 21) + 2), -1), (dict(out=(1 << 21) + 2), -1), (dict(kd=(1 << 21) + 2), -1),
    (dict(vd=(1 << 21) + 2), -1), (dict(mask=(1 << 21) + 2), -1), (dict(lse=(1 << 21) + 2), -1),
    (dict(n=0), -1), (dict(n=257), -2), (dict(tokens=(-1, 5)), -1), (dict(tokens=(5, 101)), -3),
    (dict(nodes=(5, 1)), -1), (dict(nodes=(1, -1)), -1), (dict(ws=0), -4), (dict(ws=(1 << 26) + 8), -4), (dict(ws_bytes=1000), -4),
])
def test_refusals(B, kw, code):
    assert call(B, config("kv4", 2, 8, 2, 100), **kw) == code


def test_refused_configs(B):
    assert call(B, config("kv4", 257, 2, 2, 100), tokens=[1] * 257) == -2
    assert call(B, config("kv4", 2, 8, 2, (1 << 30) + 1)) == -2
    assert call(B, config("kv4", 2, 8, 2, 100, head_dim=64)) == -2


def test_nothing_to_do(B):
    """No row holds a node: nothing is launched (and no GPU is needed)."""
    assert call(B, config("kv4", 2, 8, 2, 100), nodes=(0, 0)) == 0


def test_workspace(B):
    cfg = config("kv4", 2, 8, 2, 100)
    sizes = [B.kvq_tree_workspace(cfg, n) for n in (1, 16, 64, 256)]
    assert all(s > 0 for s in sizes) and sizes == sorted(sizes)
    for n, code in ((0, -1), (257, -2)):
        with pytest.raises(B.KvqError) as e:
            B.kvq_tree_workspace(cfg, n)
        assert e.value.status == code
    assert B.lib().kvq_tree_workspace(C.byref(B.make_config(cfg)), 4, None) == -1


def test_tree_mask(B):
    m = B.tree_mask([[-1, 0, 0, 1, -1], [-1, -1, 1, 2, 3]]).numpy()
    assert m.shape == (2, 5, 1)
    assert m[0, :, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000]
    assert m[1, :, 0].tolist() == [0b1, 0b10, 0b110, 0b1110, 0b11110]
    chain = B.tree_mask([list(range(-1, 69))]).numpy().view(np.uint32)
    assert chain.shape == (1, 70, 3) and chain[0, 69].tolist() == [0xFFFFFFFF, 0xFFFFFFFF, 0b111111]
    for bad in ([[0]], [[-1, 2]], [[-2]], [], [[]]):
        with pytest.raises(ValueError):
            B.tree_mask(bad)
