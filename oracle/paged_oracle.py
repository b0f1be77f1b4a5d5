"""The paged 8-bit cache from its definition, in numpy and 64 bits: the E4M3
codes and their power-of-two page scales, the append, attention over the
pages, and compaction.  Shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

E_MIN, E_MAX = -60, 60


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3
    fraction bits; exponent 0 is subnormal; 0x7f and 0xff are NaN."""
    v = np.empty(256)
    for c in range(256):
        s, e, f = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        v[c] = s * (f / 8.0 * 2.0 ** -6 if e == 0 else (1 + f / 8.0) * 2.0 ** (e - 7))
    v[0x7F] = v[0xFF] = np.nan
    return v


VALUES = e4m3_values()


def e4m3_round(x) -> np.ndarray:
    """Nearest E4M3 value, ties to the even code, beyond 448 to 448."""
    x = np.asarray(x, np.float64)
    mag = np.abs(x)
    with np.errstate(divide="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(mag > 0, mag, 1e-300))), -6)
    step = 2.0 ** (e - 3)
    return np.copysign(np.minimum(np.rint(mag / step) * step, 448.0), x)


def e4m3_code(v) -> np.ndarray:
    """The code of each E4M3 value (the zero of either sign by its sign)."""
    v = np.asarray(v, np.float64)
    table = {float(abs(VALUES[c])): c for c in range(0x7F)}
    codes = np.array([table[float(abs(x))] for x in v.reshape(-1)], np.uint8).reshape(v.shape)
    return np.where(np.signbit(v), codes | 0x80, codes).astype(np.uint8)


def scale_exponent(amax: float) -> int:
    """Smallest e in [-60, 60] with amax <= 448 * 2^e (60 when there is none)."""
    for e in range(E_MIN, E_MAX):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


class Pool:
    """One layer of a pool: values (not codes) [n_pages, heads, page, d] and
    scale exponents [n_pages, heads], K and V."""

    def __init__(self, codes, exps):
        self.val = [VALUES[np.asarray(c, np.uint8)] for c in codes]
        self.exp = [np.array(e, np.int64) for e in exps]
        self.page = self.val[0].shape[2]

    def rows(self, kv: int, table_row, length: int) -> np.ndarray:
        """[heads, length, d] of one sequence, in original units."""
        n = -(-length // self.page)
        ids = np.asarray(table_row[:n], np.int64)
        x = self.val[kv][ids] * 2.0 ** self.exp[kv][ids][:, :, None, None]
        return x.transpose(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :length]


def append(pool: Pool, k_new, v_new, table, lens, counts):
    """In place: counts[b] rows of sequence b end at position lens[b] - 1."""
    at = 0
    for b, (length, n) in enumerate(zip(lens, counts)):
        start = length - n
        for p in range(start // pool.page, -(-length // pool.page) if n else 0):
            lo, hi = max(start, p * pool.page), min(length, (p + 1) * pool.page)
            if lo >= hi:
                continue
            page = table[b][p]
            for kv, x in ((0, k_new), (1, v_new)):
                x = np.asarray(x, np.float64)[at + lo - start:at + hi - start]
                for h in range(x.shape[1]):
                    e = scale_exponent(np.abs(x[:, h]).max())
                    i0, i1 = lo - p * pool.page, hi - p * pool.page
                    if i0 > 0:
                        old = pool.exp[kv][page, h]
                        e = max(e, old)
                        if e > old:
                            pool.val[kv][page, h, :i0] = e4m3_round(pool.val[kv][page, h, :i0] * 2.0 ** (old - e))
                    pool.val[kv][page, h, i0:i1] = e4m3_round(x[:, h] * 2.0 ** -e)
                    pool.exp[kv][page, h] = e
        at += n


def attention(pool: Pool, q, table, lens, counts, scale: float, causal: bool, window: int):
    """(out [rows, q_heads, d], lse [rows, q_heads], bound [rows, q_heads, d],
    score_err [rows, q_heads], query_err [rows, q_heads]).  What the error of
    a lower-precision evaluation is measured by, over the attended keys:
    ``bound`` is sum_j p_j |v_j| per channel, score_err scale * max_j sum_c
    |q_c k_jc|, query_err scale * max_c |q_c| * max_j sum_c |k_jc|."""
    q = np.asarray(q, np.float64)
    rows, hq, d = q.shape
    out, lse = np.zeros((rows, hq, d)), np.full((rows, hq), -math.inf)
    bound, serr, qerr = np.zeros((rows, hq, d)), np.zeros((rows, hq)), np.zeros((rows, hq))
    at = 0
    for b, (length, n) in enumerate(zip(lens, counts)):
        k, v = pool.rows(0, table[b], length), pool.rows(1, table[b], length)
        j = np.arange(length)
        for i in range(n):
            t = length - n + i
            see = np.ones(length, bool)
            if causal:
                see &= j <= t
            if window > 0:
                see &= j > t - window
            if not see.any():
                continue
            for h in range(hq):
                g = h // (hq // k.shape[0])
                s = scale * (k[g][see] @ q[at + i, h])
                m = s.max()
                p = np.exp(s - m)
                lse[at + i, h] = m + math.log(p.sum())
                p /= p.sum()
                out[at + i, h] = p @ v[g][see]
                bound[at + i, h] = p @ np.abs(v[g][see])
                serr[at + i, h] = scale * (np.abs(k[g][see]) @ np.abs(q[at + i, h])).max()
                qerr[at + i, h] = scale * np.abs(q[at + i, h]).max() * np.abs(k[g][see]).sum(1).max()
        at += n
    return out, lse, bound, serr, qerr


def compact(table, n_pages: int):
    """(new table, number of live pages, [(from, to), ...])."""
    t = np.asarray(table)
    live = sorted(set(int(x) for x in t.reshape(-1) if x >= 0))
    n = len(live)
    holes = [i for i in range(n) if i not in set(live)]
    moves = list(zip([x for x in live if x >= n], holes))
    to = dict(moves)
    return np.vectorize(lambda x: to.get(int(x), int(x)))(t) if t.size else t, n, moves


def rope(x, positions, frequency, axis, interleaved: bool, inverse: bool = False):
    """Rows x [rows, heads, d] turned by their positions [rows, axes]: pair p, of
    the axis axis[p], by the angle position * frequency[p]."""
    x = np.array(x, np.float64)
    n = len(frequency)
    angle = np.asarray(positions, np.float64)[:, np.asarray(axis)] * np.asarray(frequency, np.float64)
    turn = np.exp((-1j if inverse else 1j) * angle)[:, None]
    first, second = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    z = (first + 1j * second) * turn
    y = x.copy()
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    else:
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y


def rope_steps(x, cos_sin, positions, axis, interleaved: bool, inverse: bool = False):
    """The same with a table [positions, pairs, 2], each product and each sum
    rounded to fp32 by itself: the values that the append quantizes."""
    x, cos_sin = np.array(x, np.float32), np.asarray(cos_sin, np.float32)
    n = cos_sin.shape[1]
    cs = cos_sin[np.asarray(positions)[:, np.asarray(axis)], np.arange(n)][:, None]
    c, s = cs[..., 0], -cs[..., 1] if inverse else cs[..., 1]
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    first, second, y = x[..., a], x[..., b], x.copy()
    y[..., a] = first * c - second * s
    y[..., b] = second * c + first * s
    return y


def attention_scored(pool: Pool, q, table, lens, counts, scale: float, causal: bool, window: int, softcap: float = 0.0,
                     slopes=None, prefix=None, ranges=None):
    """attention with shaped scores and further masks: what it returns, and
    last shape_err [rows, q_heads], max_j of |s_j| + |bias_j|, by which the
    rounding of the shaping itself is measured, and top [rows, q_heads], the
    largest product of a weight and its V scale."""
    q = np.asarray(q, np.float64)
    rows, hq, d = q.shape
    out, lse = np.zeros((rows, hq, d)), np.full((rows, hq), -math.inf)
    bound, serr, qerr, herr = np.zeros((rows, hq, d)), np.zeros((rows, hq)), np.zeros((rows, hq)), np.zeros((rows, hq))
    tops = np.zeros((rows, hq))
    at = 0
    for b, (length, n) in enumerate(zip(lens, counts)):
        k, v = pool.rows(0, table[b], length), pool.rows(1, table[b], length)
        ev = 2.0 ** np.repeat(pool.exp[1][np.asarray(table[b][:-(-length // pool.page)], np.int64)], pool.page, axis=0)[:length]
        j = np.arange(length)
        for i in range(n):
            t = length - n + i
            see = np.ones(length, bool)
            if causal:
                see &= (j <= t) | (j < (0 if prefix is None else int(prefix[b])))
            if window > 0:
                see &= j > t - window
            if ranges is not None:
                see &= (j >= int(ranges[at + i][0])) & (j < int(ranges[at + i][1]))
            if not see.any():
                continue
            for h in range(hq):
                g = h // (hq // k.shape[0])
                s = scale * (k[g][see] @ q[at + i, h])
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                bias = 0 * s if slopes is None else -float(slopes[h]) * np.abs(t - j[see])
                herr[at + i, h] = (np.abs(s) + np.abs(bias)).max()
                s = s + bias
                m = s.max()
                p = np.exp(s - m)
                lse[at + i, h] = m + math.log(p.sum())
                p /= p.sum()
                out[at + i, h] = p @ v[g][see]
                bound[at + i, h] = p @ np.abs(v[g][see])
                tops[at + i, h] = (p * ev[see, g]).max()
                serr[at + i, h] = scale * (np.abs(k[g][see]) @ np.abs(q[at + i, h])).max()
                qerr[at + i, h] = scale * np.abs(q[at + i, h]).max() * np.abs(k[g][see]).sum(1).max()
        at += n
    return out, lse, bound, serr, qerr, herr, tops
