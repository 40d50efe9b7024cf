"""The block attention's bounds (_block_bounds.py) on the host: the result in 64 bits, rounded,
passes; one with a mistake planted in it does not."""
import numpy as np
import pytest

pytest.importorskip("torch")

from tests._block_bounds import BLOCK, Request, ends, naming, parts_of, two_level  # noqa: E402
from tests._block_testutil import D  # noqa: E402
from tests.test_gpu_block_attn import Pool  # noqa: E402

SCALE = 1 / np.sqrt(D)


def inside(pool, planted=None, weights=None, position=None):
    """Whether the last token's rows pass, with other values or weights in the result."""
    length, good = pool.lens[0], True
    r = Request(pool.codes, pool.scales, pool.table[0], length)
    v = r.c * 2.0 ** r.ev[..., None]
    v2 = v.copy()
    if planted is not None:
        planted(v2)
    g = pool.hq // pool.hkv
    for h in range(pool.hq):
        o, err, a, tiny, *_ = r.row(pool.q[-1, h], h // g, length - 1, SCALE)
        lo, hi = ends(o, err, a, tiny, parts_of(pool.cfg))
        w = r.row(pool.q[-1, h], h // g, length - 1, SCALE, v=v2, weights=weights)[0]
        got = w.astype(np.float16).astype(float)
        good &= bool(((lo.astype(float) <= got) & (got <= hi.astype(float))).all())
    return good


def no_block(j):
    def f(v):
        v[:, j * BLOCK:(j + 1) * BLOCK] = 0
    return f


def no_row(t):
    def f(v):
        v[:, t] = 0
    return f


def swapped(t):
    def f(v):
        v[:, [t, t + 1]] = v[:, [t + 1, t]]
    return f


def shifted(j):
    """A block's rows one place on."""
    def f(v):
        v[:, j * BLOCK:(j + 1) * BLOCK] = np.roll(v[:, j * BLOCK:(j + 1) * BLOCK], 1, 1)
    return f


def heaviest(pool, size):
    """In each third of the context the run of `size` tokens (from a multiple of it) that has
    the most weight in the first head's last row."""
    length = pool.lens[0]
    r = Request(pool.codes, pool.scales, pool.table[0], length)
    z = SCALE * (r.k[0] @ pool.q[-1, 0].astype(float))
    w = np.exp(z - z.max())
    w = w[:length // size * size].reshape(-1, size).sum(1)
    return [int(np.argmax(x)) + at for x, at in zip(np.array_split(w, 3), np.cumsum([0] + [len(x) for x in np.array_split(w, 3)]))]


@pytest.mark.parametrize("new", [1, 4])  # two parts of a weight, one
@pytest.mark.parametrize("length", [96, 700, 9000])
def test_random_values(length, new):
    p = Pool([length], [new], 4, 1, seed=length)
    assert inside(p)
    for j in heaviest(p, BLOCK):
        assert not inside(p, no_block(j)) and not inside(p, shifted(j)), j
    for t in heaviest(p, 1):
        assert not inside(p, no_row(t)), t
        assert not inside(p, swapped(min(t, length - 2))), t


@pytest.mark.parametrize("new", [1, 4])
@pytest.mark.parametrize("length", [300, 3000, 12000])
def test_values_that_name_their_tokens(length, new):
    p = Pool([length], [new], 4, 1, seed=1)
    naming(p)
    assert inside(p)
    for t in (0, 31, 32, length // 2, length - 2):
        assert not inside(p, no_row(t)), t
        assert not inside(p, swapped(t)), t
    for j in (0, length // 64, length // 32 - 1):
        assert not inside(p, no_block(j)) and not inside(p, shifted(j)), j


def one_part(w):
    return (w * 2.0**12).astype(np.float16).astype(float) * 2.0**-12


def two_parts(w):
    w = w * 2.0**12
    h = w.astype(np.float16).astype(float)
    return (h + (w - h).astype(np.float16).astype(float)) * 2.0**-12


@pytest.mark.parametrize("length", [64, 1000])
def test_parts_of_a_weight(length):
    """Up to 8 rows the weights have 22 bits: one fp16 part falls outside."""
    p = Pool([length], [1], 4, 1, seed=2)
    assert abs(two_level(p)) > 0.9 * 2.0**-11
    assert inside(p, weights=two_parts) and not inside(p, weights=one_part)
    q = Pool([length], [4], 4, 1, seed=2)  # 16 rows
    two_level(q)
    assert parts_of(q.cfg) == 1 and inside(q, weights=one_part)
