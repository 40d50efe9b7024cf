"""Tensors whose shape does not match the call are refused: read with the
call's strides they would give a wrong result without an error."""
import pytest
import torch

from _spec_testutil import config


def test_which_shapes_fit():
    from bit_kv_cache_07_gb300.binding import _fits
    want = (2, 8, 5, 128)
    for shape in (want, (4, 8, 5, 128), (16, 5, 128), (2 * 8 * 5 * 128,), (99999999,), (2, 8, 1, 5, 128)):
        assert _fits(torch.Size(shape), want), shape
    for shape in ((2, 8, 6, 128), (2, 5, 8, 128), (2, 9, 5, 128), (2, 8, 5, 256), (16, 6, 128), (3, 16, 5, 128)):
        assert not _fits(torch.Size(shape), want), shape
    assert _fits((2, 8), (2, 8, 1)) and not _fits((2, 8, 4), (2, 8, 1))


@pytest.fixture(scope="module")
def B():
    from bit_kv_cache_07_gb300 import build
    build.build_library()
    from bit_kv_cache_07_gb300 import binding
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return binding


def zeros(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


@pytest.mark.gpu
def test_refused_shapes(B):
    cfg = config("kv4", 2, 4, 2, 300)
    layer, f = B.Layer(cfg), torch.float32
    layer.append(0, zeros(2, 2, 200, 128), zeros(2, 2, 200, 128))
    q, out, kv, words = zeros(2, 4, 3, 128), zeros(2, 4, 3, 128), zeros(2, 2, 3, 128), B.tree_mask([[-1, 0, 1]] * 2).cuda()
    lse, ws, mass, ews = zeros(2, 4, 3, dtype=f), B.new_tree_workspace(cfg, 8), B.new_mass(cfg), B.new_evict_workspace(cfg)
    good = dict(q=q, k=kv, v=kv, mask=words, out=out, lse=lse)

    def tree(**kw):
        a = dict(good, **kw)
        layer.tree_attn([200, 100], a["q"], a["k"], a["v"], a["mask"], a["out"], a["lse"], ws)

    for bad in (dict(q=zeros(2, 3, 4, 128)), dict(q=zeros(2, 4, 3, 256)), dict(k=zeros(2, 2, 8, 128)), dict(v=zeros(2, 2, 8, 128)),
                dict(v=zeros(2, 3, 2, 128)), dict(mask=zeros(2, 3, 2, dtype=torch.int32)), dict(mask=zeros(2, 8, 1, dtype=torch.int32)),
                dict(out=zeros(2, 4, 8, 128)), dict(out=zeros(2, 3, 4, 128)), dict(lse=zeros(2, 4, 8, dtype=f))):
        with pytest.raises(ValueError):
            tree(**bad)

    def record(q=q, lse=lse, mass=mass, weight=None):
        layer.attn_mass([200, 100], q, lse, mass, weight)

    for bad in (dict(lse=zeros(2, 4, 8, dtype=f)), dict(mass=zeros(2, 2, 400, dtype=f)), dict(mass=zeros(2, 4, 300, dtype=f)),
                dict(weight=zeros(2, 8, dtype=f)), dict(q=zeros(2, 4, 128))):
        with pytest.raises(ValueError):
            record(**bad)
    for bad in (dict(mass=zeros(2, 2, 400, dtype=f)), dict(out=zeros(2, 3, 300, dtype=f)), dict(source=zeros(2, 2, 9, dtype=torch.int32))):
        a = dict(dict(mass=mass, out=mass, source=None), **bad)
        with pytest.raises(ValueError):
            layer.evict([200, 100], [1, 1], a["mass"], a["out"], a["source"], ews)

    # what is read right stays accepted: flat buffers, more rows behind the batch, a decode's q and lse
    tree(out=zeros(2 * 4 * 3 * 128 + 64), lse=zeros(3, 4, 3, dtype=f), mask=words.view(2, 3))
    record(q=zeros(2, 4, 128), lse=zeros(2, 4, dtype=f))
    record(mass=mass.view(-1), weight=torch.ones(2, 3, device="cuda"))
    torch.cuda.synchronize()
