"""What a row of the block attention may be off by, from the row's own terms: an interval
of fp16 numbers around the result in 64 bits, narrow enough that a value block left out,
one value row left out or two exchanged fall outside of it.

For a row with weights p_t (of sum 1), values v_t = c_t 2^ev_t, o = sum p_t v_t,
A = sum p_t |v_t| (by channel):
- logits: fp32 sums of 128 products in 8 steps of 16, each step's additions off by less
  than 4 * 2^-24 of the terms so far: 2^-19 scale sum |q_i k_ti|; the exponent's
  argument passes three fp32 roundings of numbers below |ev_t| + 1.5 |max logit| + 32
  (bits); the exponential itself, and those that move a reference or join two parts
  (a few each), 2^-20 together: e_t.  A weight that is off by e_t moves o by p_t
  (v_t - o) e_t.
- weights enter the product in fp16: 2^-11 of each in one part, 2^-22 in two, and no
  finer than half of fp16's least step, 2^-25, where the largest p_t 2^ev_t, u, stands
  at 2^12 or more: 2^-37 u |c_t|.
- sums of products and of weights: below 64 additions one after the other per warp at
  the sizes of these tests, each off by less than 2 * 2^-24 of the terms: 2^-17 of A and
  of |o|.
The result is rounded once to fp16, which is monotone: out lies between the rounded
ends of o +- that sum.  lse: sum p_t e_t, the sum's 2^-17, and fp32 steps of the
logarithm and of numbers up to its parts."""
import numpy as np

from tests._block_testutil import BLOCK, D, E4M3, unswizzled


def seen(length, p, window, first):
    t = np.arange(length)
    s = t <= p
    return s & ((p - t < window) | (t < first)) if window else s


class Request:
    """A request's keys, values and value exponents in 64 bits, read from its blocks once."""

    def __init__(self, codes, scales, table, length):
        ids = np.asarray(table[:-(-length // BLOCK)])
        c = E4M3[unswizzled(codes[ids])].transpose(1, 2, 0, 3, 4).reshape(codes.shape[1], 2, -1, D)[:, :, :length]
        e = (scales[ids].astype(float) - 127).transpose(1, 2, 0).repeat(BLOCK, 2)[:, :, :length]
        self.k, self.c, self.ev, self.length = c[:, 0] * 2.0 ** e[:, 0, :, None], c[:, 1], e[:, 1], length

    def row(self, q, head, p, scale, window=0, first=0, v=None, weights=None):
        """(out, its error, lse, its error) of query q at position p; v: other values than the
        request's; weights: what becomes of exp(z - max) before it meets the values."""
        s = seen(self.length, p, window, first)
        k, c, ev = self.k[head][s], self.c[head][s], self.ev[head][s]
        v = (c * 2.0 ** ev[:, None]) if v is None else v[head][s]
        q = q.astype(np.float64)
        z = scale * (k @ q)
        m = z.max()
        w = np.exp(z - m)
        l = w.sum()
        p_t = w / l
        out = (p_t if weights is None else weights(w) / l) @ v
        e = 2.0**-19 * scale * (np.abs(k) @ np.abs(q)) + 2.0**-23 * (np.abs(ev) + 1.5 * abs(m) + 32) + 2.0**-20
        a = p_t @ np.abs(v)
        err = p_t @ (np.abs(v) * e[:, None]) + (p_t @ e) * np.abs(out) + 2.0**-17 * (a + np.abs(out))
        u = (p_t * 2.0**ev).max()
        tiny = 2.0**-37 * u * np.abs(c).sum(0)
        lse = m + np.log(l)
        return out, err, a, tiny, lse, p_t @ e + 2.0**-17 + 2.0**-22 * (abs(lse) + np.abs(ev).max() + 32)


def ends(out, err, a, tiny, parts):
    """The fp16 numbers between which a row lies; parts: fp16 parts of a weight."""
    d = err + tiny + a * (2.0**-22 if parts == 2 else 2.0**-11)
    with np.errstate(over="ignore"):
        return (out - d).astype(np.float16), (out + d).astype(np.float16)


def parts_of(cfg):
    """Two up to 8 rows of a KV head in an even share of the token slots."""
    g = cfg["n_q_heads"] // cfg["n_kv_heads"]
    return 2 if -(-cfg["n_tokens"] // cfg["batch"]) * g <= 8 else 1


def check(pool, out, lse, rows=None):
    """Every row (or the chosen token slots' rows) of a Pool's results within its interval."""
    cfg, at, g = pool.cfg, 0, pool.hq // pool.hkv
    scale = cfg.get("softmax_scale") or 1 / np.sqrt(D)
    for b, (length, n) in enumerate(zip(pool.lens, pool.new)):
        r = Request(pool.codes, pool.scales, pool.table[b], length)
        for i in range(n):
            if rows is not None and at + i not in rows:
                continue
            for h in range(pool.hq):
                o, err, a, tiny, s, s_err = r.row(pool.q[at + i, h], h // g, length - n + i, scale, cfg.get("window", 0), cfg.get("n_first", 0))
                lo, hi = ends(o, err, a, tiny, parts_of(cfg))
                got = out[at + i, h]
                ok = (lo.astype(float) <= got) & (got <= hi.astype(float))
                assert ok.all(), (b, i, h, int((~ok).sum()), float(np.max(np.abs(got - o) / (err + tiny + np.abs(o) * 2.0**-11 + 2.0**-25))))
                assert abs(lse[at + i, h] - s) <= s_err, (b, i, h, lse[at + i, h] - s, s_err)
        at += n


def two_level(pool):
    """Makes a Pool's logits take two values, which meet in every block: token 0's is the
    larger and its value zero; the others' weight rounds to one fp16 part with nearly the
    largest error, always in the same direction, so that out is off by as much."""
    scale = pool.cfg.get("softmax_scale") or 1 / np.sqrt(D)
    best, best_q = 0.0, 1.0
    for q0 in np.arange(4.0, 9.0, 2.0**-8):  # fp16 numbers
        w = 2.0**12 * np.exp(-scale * q0)  # keys 1 and 0, the larger at 2^12
        err = (float(np.float16(w)) - w) / w
        if abs(err) > abs(best):
            best, best_q = err, q0
    pool.q[:] = 0
    pool.q[..., 0] = best_q
    pool.codes[:, :, 0] = 0
    pool.codes[:, :, 0, 0, 0] = 0x38  # 1.0, channel 0 of token 0 (chunk 0 lies at 0 ^ 0)
    pool.scales[:] = 127
    pool.codes[:, :, 1] &= 0x7F  # values of one sign, moderate
    pool.codes[:, :, 1] = np.clip(pool.codes[:, :, 1], 0x20, 0x40)
    pool.codes[:, :, 1, 0] = 0  # token 0's values
    return best


def naming(pool):
    """Makes a Pool's values name their tokens: token t has a one at channel 37 t + 5 t // 128
    (mod 128) and nothing else; weights differ by up to four times from token to token."""
    pool.q[:] = 0
    pool.q[..., 0] = 8.0
    pool.scales[:] = 127
    pool.codes[:] = 0
    for b, length in enumerate(pool.lens):
        t = np.arange(length)
        blk, row = pool.table[b][t // BLOCK], t % BLOCK
        ch = (37 * t + 5 * (t // 128)) % D
        for h in range(pool.hkv):
            pool.codes[blk, h, 1, row, ((ch // 16) ^ (row % 8)) * 16 + ch % 16] = 0x38
            pool.codes[blk, h, 0, row, (row % 8) * 16] = 0x28 + (t * 7 + h) % 24  # 2^-2 .. 2
