"""Shared helpers of the block cache's tests: the e4m3 format, the plan, the append
and the attention in plain Python and numpy, in 64 bits, request by request."""
from __future__ import annotations

import numpy as np

D, BLOCK = 128, 32
EPS = 1e-6

# the values of the 256 e4m3 bytes, from the format's definition
_b = np.arange(256)
_exp, _man = (_b >> 3) & 15, _b & 7
E4M3 = np.where(_exp == 0, _man / 8.0 * 2.0**-6, (1 + _man / 8.0) * 2.0 ** (_exp - 7.0))
E4M3 = np.where((_b & 127) == 127, np.nan, np.where(_b > 127, -E4M3, E4M3))


def half_step(y):
    """Half the distance of neighbouring e4m3 values around |y| <= 448 (steps are
    2^-3 of the power of two below, 2^-9 under 2^-6)."""
    y = np.maximum(np.abs(y), 2.0**-6)
    return 2.0 ** (np.floor(np.log2(y)) - 4)


def unswizzled(block):
    """[..., 32, 128] stored bytes -> the rows' channels in order."""
    t = np.arange(BLOCK)[:, None]
    chunk = np.arange(8)[None] ^ (t % 8)
    rows = block.reshape(block.shape[:-1] + (8, 16))
    return np.take_along_axis(rows, np.broadcast_to(chunk[..., None], rows.shape), axis=-2).reshape(block.shape)


def values(codes, scales):
    """Stored keys and values [n_blocks, H, 2, 32, 128] in 64 bits."""
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return E4M3[unswizzled(codes)] * s[..., None, None]


def normed_rotated(x, weight, pos, theta, eps=EPS):
    """x [n, H, 128] fp16 -> 64 bits."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * weight.astype(np.float64)
    if theta:
        f = float(np.float32(theta)) ** (-2.0 * np.arange(64) / D)
        a = np.asarray(pos, np.float64)[:, None] * f
        z = (x[..., :64] + 1j * x[..., 64:]) * np.exp(1j * a)[:, None]
        x = np.concatenate([z.real, z.imag], -1)
    return x


def exponent(amax):
    """The least e in [-40, 40] with amax <= 448 * 2^e."""
    e = -40
    while e < 40 and amax > 448.0 * 2.0**e:
        e += 1
    return e


class Plan:
    """kvq_block_plan, request by request."""

    def __init__(self, batch, n_tokens, n_blocks, max_blocks):
        self.B, self.N, self.nb, self.M = batch, n_tokens, n_blocks, max_blocks
        self.lens = [0] * batch
        self.table = np.zeros((batch, max_blocks), np.int32)
        self.stack = list(range(n_blocks - 1, -1, -1))
        self.free = n_blocks

    def step(self, n_new):
        before = list(self.lens)
        held = [-(-l // BLOCK) for l in before]
        for b, n in enumerate(n_new):
            if n < 0:
                for j in range(held[b]):
                    self.stack[self.free] = int(self.table[b, j])
                    self.free += 1
        total, asked, tokens = self.free, 0, 0
        start, unit0, row, pos, slot = [0], [0], [], [], []
        for b, n in enumerate(n_new):
            l, took = before[b], 0
            if n < 0:
                self.lens[b] = 0
            elif l + n <= self.M * BLOCK:
                need = -(-(l + n) // BLOCK) - held[b]
                asked, tokens = asked + need, tokens + n
                if (need == 0 or asked <= total) and tokens <= self.N:
                    took = n
                    for j in range(held[b], held[b] + need):
                        self.free -= 1
                        self.table[b, j] = self.stack[self.free]
                    self.lens[b] = l + n
            start.append(start[-1] + took)
            unit0.append(unit0[-1] + (-(-(l + took) // BLOCK) - l // BLOCK if took else 0))
            for p in range(l, l + took):
                row.append(b)
                pos.append(p)
                slot.append(int(self.table[b, p // BLOCK]) * BLOCK + p % BLOCK)
        pad = self.N - len(row)
        self.start, self.unit0 = start, unit0
        self.row, self.pos, self.slot = row + [-1] * pad, pos + [0] * pad, slot + [-1] * pad
        return self

    def same(self, t):
        """Whether the GPU's tables t are these."""
        n = lambda x: x.cpu().numpy()  # noqa: E731
        assert n(t.lens).tolist() == self.lens
        assert n(t.start).tolist() == self.start and n(t.unit0).tolist() == self.unit0
        assert n(t.token_row).tolist() == self.row and n(t.position).tolist() == self.pos
        assert n(t.slot).tolist() == self.slot
        assert int(t.free_count) == self.free
        assert n(t.free_list).tolist() == self.stack
        assert np.array_equal(n(t.block_table), self.table)


def attention(q, kv, table, length, n, hq, hkv, window=0, first=0, scale=None):
    """q [n, Hq, 128] at the last n of `length` positions over the values kv
    (see `values`) of a request's blocks: (out, lse) in 64 bits."""
    g = hq // hkv
    ids = np.asarray(table[:-(-length // BLOCK)])
    k = kv[ids, :, 0].transpose(1, 0, 2, 3).reshape(hkv, -1, D)[:, :length]
    v = kv[ids, :, 1].transpose(1, 0, 2, 3).reshape(hkv, -1, D)[:, :length]
    out, lse = np.zeros((n, hq, D)), np.zeros((n, hq))
    scale = 1 / np.sqrt(D) if scale is None else scale
    t = np.arange(length)
    for i in range(n):
        p = length - n + i
        sees = t <= p
        if window:
            sees &= (p - t < window) | (t < first)
        for h in range(hq):
            z = scale * (k[h // g][sees] @ q[i, h].astype(np.float64))
            m = z.max() if not np.isnan(z).any() else np.nan
            e = np.exp(z - m)
            lse[i, h] = m + np.log(e.sum())
            out[i, h] = e @ v[h // g][sees] / e.sum()
    return out, lse
