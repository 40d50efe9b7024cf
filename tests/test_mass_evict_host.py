"""Refusals of kvq_attn_mass, kvq_evict and kvq_evict_workspace without a GPU:
every bad argument is returned before anything is launched."""
import ctypes as C
import math

import pytest

from _spec_testutil import config


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    return binding


def arr(v):
    return None if v is None else (C.c_int32 * len(v))(*v)


def mass(B, cfg, tokens=(10, 20), n=4, decay=1.0, **kw):
    a = dict(layer=1 << 20, q=1 << 21, lse=1 << 22, weight=0, mass=1 << 23)
    a.update(kw)
    return B.lib().kvq_attn_mass(C.byref(B.make_config(cfg)), a["layer"] or None, arr(tokens), a["q"] or None, a["lse"] or None,
                                 a["weight"] or None, n, decay, a["mass"] or None, None)


def evict(B, cfg, tokens=(200, 100), drop=(1, 0), **kw):
    a = dict(layer=1 << 20, mass=1 << 24, out=1 << 24, source=0, ws=1 << 26, ws_bytes=1 << 40)
    a.update(kw)
    return B.lib().kvq_evict(C.byref(B.make_config(cfg)), a["layer"] or None, arr(tokens), arr(drop), a["mass"] or None,
                             a["out"] or None, a["source"] or None, a["ws"] or None, a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(layer=0), -1), (dict(q=0), -1), (dict(lse=0), -1), (dict(mass=0), -1), (dict(tokens=None), -1),
    (dict(layer=(1 << 20) + 4), -1), (dict(q=(1 << 21) + 8), -1), (dict(lse=(1 << 21) + 2), -1), (dict(weight=(1 << 21) + 1), -1),
    (dict(mass=(1 << 21) + 2), -1), (dict(n=0), -1), (dict(n=(1 << 20) + 1), -2), (dict(decay=math.inf), -1),
    (dict(decay=math.nan), -1), (dict(tokens=(-1, 0)), -1), (dict(tokens=(0, 101)), -3),
])
def test_mass_refusals(B, kw, code):
    assert mass(B, config("kv4", 2, 8, 2, 100), **kw) == code


def test_mass_of_empty_rows(B):
    assert mass(B, config("kv4", 2, 8, 2, 100), tokens=(0, 0)) == 0
    assert mass(B, config("kv4", 257, 2, 2, 100), tokens=[0] * 257) == -2


@pytest.mark.parametrize("kw,code", [
    (dict(layer=0), -1), (dict(mass=0), -1), (dict(out=0), -1), (dict(tokens=None), -1), (dict(drop=None), -1),
    (dict(layer=(1 << 20) + 8), -1), (dict(mass=(1 << 24) + 2), -1), (dict(source=(1 << 24) + 2), -1),
    (dict(out=(1 << 24) + 64), -1), (dict(out=(1 << 24) - 64), -1),  # half over the input record
    (dict(ws=0), -4), (dict(ws=(1 << 26) + 8), -4), (dict(ws_bytes=64), -4),
    (dict(tokens=(-1, 0)), -1), (dict(tokens=(301, 0)), -3), (dict(drop=(-1, 0)), -1),
    (dict(drop=(6, 0)), -1), (dict(drop=(5, 3)), -1), (dict(tokens=(35, 0), drop=(1, 0)), -1),
])
def test_evict_refusals(B, kw, code):
    # (200 - 36) / 32 = 5 groups and (100 - 36) / 32 = 2 groups at most
    assert evict(B, config("kv4", 2, 8, 2, 300), **kw) == code


def test_evict_refused_configs(B):
    for form, more, code in (("kv4_rope", {}, -2), ("fp16_rope", {}, -2), ("nuq_rope", {}, -2), ("kv4", dict(head_dim=64), -2)):
        cfg = config(form, 2, 8, 2, 300, **more)
        assert evict(B, cfg) == code
        with pytest.raises(B.KvqError) as e:
            B.kvq_evict_workspace(cfg)
        assert e.value.status == code
    assert evict(B, config("kv4", 257, 2, 2, 300), tokens=[0] * 257, drop=[0] * 257) == -2
    assert B.lib().kvq_evict_workspace(C.byref(B.make_config(config("kv4", 2, 8, 2, 300))), None) == -1


def test_workspace_sizes(B):
    small, large = (B.kvq_evict_workspace(config("kv4", 2, 8, 2, t)) for t in (300, 30000))
    assert 0 < small < large
    assert B.kvq_evict_workspace(config("fp16", 2, 8, 2, 20)) >= 0  # no group fits
