"""kvq_block_plan against the request-by-request model: prompts, tokens, ends,
refusals, unused slots, repeated and captured calls, tables out of range."""
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_kv_cache_07_gb300 import blocks  # noqa: E402
from tests._block_testutil import BLOCK, Plan  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_07_gb300 import build
    build.build_library()


def make(batch, n_tokens, n_blocks, max_blocks, **arrays):
    return blocks.Tables(dict(batch=batch, n_tokens=n_tokens, n_q_heads=1, n_kv_heads=1, head_dim=128, n_blocks=n_blocks,
                              max_blocks=max_blocks), **arrays)


def dev(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# one request to the most, one thread's slots and several CTAs', pools that run out
@pytest.mark.parametrize("batch,n_tokens,n_blocks,max_blocks", [
    (1, 1, 1, 1), (1, 40, 3, 2), (3, 64, 7, 4), (16, 16, 40, 9), (33, 1500, 60, 8), (64, 64, 64, 64), (200, 5000, 300, 20),
    (1024, 9000, 700, 12), (1000, 1024, 5000, 5)])
def test_steps(batch, n_tokens, n_blocks, max_blocks):
    r = random.Random(batch * 7 + n_tokens)
    model, t = Plan(batch, n_tokens, n_blocks, max_blocks), make(batch, n_tokens, n_blocks, max_blocks)
    for _ in range(12):
        few = max(1, n_tokens // batch)
        new = [r.choice([0, 1, 1, 1, -1, r.randrange(0, 2 * few + 2), r.randrange(0, BLOCK * max_blocks + 2)]) for _ in range(batch)]
        t.plan(dev(new))
        model.step(new).same(t)


def test_refused_for_want_of_blocks_only_then():
    """A request that finds no block leaves those that need none served."""
    model, t = Plan(3, 200, 4, 4), make(3, 200, 4, 4)
    for new in ([33, 31, 1], [60, 1, 100], [0, 0, 31], [0, 1, 1], [-1, 1, 1], [40, -5, -1], [128, 1, 1], [1, 0, 0]):
        t.plan(dev(new))
        model.step(new).same(t)


def test_lengths_apart_from_the_tables():
    """With lengths and count of their own the call can be repeated."""
    model, t = Plan(5, 300, 30, 6), make(5, 300, 30, 6)
    first = [10, 64, 0, 33, 5]
    t.plan(dev(first))
    model.step(first)
    lens, count = t.lens.clone(), t.free_count.clone()
    new = [1, 1, 40, -1, 70]
    model.step(new)
    for _ in range(3):
        t.plan(dev(new), lens=lens, free_count=count)
        model.same(t)


def test_captured():
    model, t = Plan(6, 100, 20, 5), make(6, 100, 20, 5)
    new = torch.zeros(6, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        t.plan(new)  # no tokens: nothing changes
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            t.plan(new)
    torch.cuda.current_stream().wait_stream(side)
    for step in ([5, 0, 33, 1, 0, 7], [1] * 6, [-1, 64, 1, 1, -1, 1], [32, 1, 1, 90, 3, 1]):
        new.copy_(dev(step))
        graph.replay()
        model.step(step).same(t)


def test_lengths_out_of_range_get_nothing():
    t = make(4, 50, 10, 3)
    lens = dev([-5, 97, 32, 2**31 - 1])
    t.plan(dev([1, 1, 1, 2**31 - 1]), lens=lens)
    assert t.lens.tolist() == [-5, 97, 33, 2**31 - 1] and t.start.tolist() == [0, 0, 0, 1, 1]
    t.plan(dev([-1, -1, 2**31 - 1, -1]))
    assert t.lens.tolist() == [0, 0, 33, 0] and int(t.free_count) == 9


def test_counts_out_of_range():
    """A free count that the stack cannot have is cut to it; nothing is written behind the stack."""
    room = torch.full((12,), 77, dtype=torch.int32, device="cuda")
    room[:10] = dev(list(range(10)))
    t = make(2, 50, 10, 3, free_list=room[:10])
    t.plan(dev([40, 1]), free_count=dev([1000]))
    assert int(t.free_count) == 7 and t.block_table[0, :2].tolist() == [9, 8] and int(t.block_table[1, 0]) == 7
    t.plan(dev([-1, -1]), free_count=dev([10]))
    assert int(t.free_count) == 10 and room[10:].tolist() == [77, 77]


def test_refused_tensors():
    t = make(4, 50, 10, 3)
    for bad in (torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda"),
                torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int32, device="cuda")[::2], [1, 1, 1, 1]):
        with pytest.raises(ValueError):
            t.plan(bad)
    with pytest.raises(ValueError):
        make(4, 50, 10, 3, lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        make(4, 50, 10, 3, lenses=torch.zeros(4, dtype=torch.int32, device="cuda"))
