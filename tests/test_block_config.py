"""The block cache's Python objects keep what their arrays were made for, whatever
the caller does with the configuration and the attributes afterwards."""
import pytest

torch = pytest.importorskip("torch")

from bit_kv_cache_07_gb300 import blocks  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


CFG = dict(batch=2, n_tokens=4, n_q_heads=4, n_kv_heads=2, head_dim=128, n_blocks=6, max_blocks=3, window=0)


def test_a_configuration_is_copied():
    c = blocks.make_config(CFG)
    d = blocks.make_config(c)
    c.n_tokens, c.window = 1 << 20, 5
    assert (d.n_tokens, d.window) == (4, 0)


@pytest.mark.gpu
def test_a_configuration_written_to_afterwards():
    """One configuration object for several layers: the first keeps its window, the
    tables their sizes (a plan of more token slots would be written behind them)."""
    c = blocks.make_config(CFG)
    t, wide = blocks.Tables(c), blocks.Layer(c)
    c.window = 1
    narrow = blocks.Layer(c)
    t.plan(torch.tensor([3, 1], dtype=torch.int32, device="cuda"))
    k, q = torch.randn((4, 2, 128), device="cuda").half(), torch.randn((4, 4, 128), device="cuda").half()
    ws, out = blocks.new_workspace(c), {}
    for name, layer in (("wide", wide), ("narrow", narrow)):
        layer.append(t, k, k.clone())
        out[name] = torch.zeros_like(q)
        layer.attn(t, q, out[name], None, ws)
    assert torch.equal(out["wide"][0], out["narrow"][0]) and not torch.equal(out["wide"][2], out["narrow"][2])
    c.n_tokens, c.batch, c.max_blocks = 4096, 64, 100
    t.plan(torch.tensor([-1, 1], dtype=torch.int32, device="cuda"))
    assert t.lens.tolist() == [0, 2] and t.start.tolist() == [0, 0, 1] and t.token_row.tolist() == [1, -1, -1, -1]


@pytest.mark.gpu
def test_tensors_are_not_exchanged():
    """The calls hold the tensors' addresses: an assignment is refused, writing in place works."""
    t, layer = blocks.Tables(CFG), blocks.Layer(CFG)
    for obj, names in ((t, ("block_table", "free_list", "free_count", "lens", "start", "unit0", "token_row", "position", "slot")),
                       (layer, ("codes", "scales"))):
        for name in names:
            old = getattr(obj, name)
            with pytest.raises(AttributeError):
                setattr(obj, name, old.clone())
            assert getattr(obj, name) is old
        obj.cfg.batch = 1000  # of a copy
        assert obj.cfg.batch == 2
    t.lens += 5
    t.free_count -= 1
    t.plan(torch.tensor([1, 0], dtype=torch.int32, device="cuda"))
    assert t.lens.tolist() == [6, 5] and int(t.free_count) == 5


@pytest.mark.gpu
def test_a_workspace_of_another_type_is_refused():
    t, layer = blocks.Tables(CFG), blocks.Layer(CFG)
    q = torch.zeros((4, 4, 128), dtype=torch.float16, device="cuda")
    ws = blocks.new_workspace(CFG)
    for bad in (ws.data_ptr(), [0] * 16, ws.cpu(), ws.int(), ws[::2]):
        with pytest.raises(ValueError):
            layer.attn(t, q, torch.zeros_like(q), None, bad)
    layer.attn(t, q, torch.zeros_like(q), None, ws)
