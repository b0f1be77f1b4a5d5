"""Paged attention over pages whose value scales lie far apart: the answer is
the formula's wherever the softmax puts its weight, on pages of large or small
scale, whatever other rows see, in every form and over the whole range of
exponents."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from quantized_kv_cache_quantize_gb300 import kvq
from tests.paged_common import cache_of, dev, offsets_of, random_pool, tolerances

pytestmark = pytest.mark.gpu

LN2 = math.log(2.0)      # the scale of these calls: a score is a number of binades


def build(seed, page, d, kv_heads, seqs, share=1.0):
    """A pool for sequences given as lists of (V exponent, score, ...) per
    page: key j of a page scores `score` binades for a query row whose first
    channel is 1 and the opposite for one whose first channel is -1; a tuple of
    scores gives them key by key (a score is rounded to an E4M3 value).  The
    pages no table names hold NaN.  Returns (cache, pool, table, scores of
    each sequence as they are)."""
    rng = np.random.default_rng(seed)
    n_pages = sum(map(len, seqs)) + 3
    codes, exps = random_pool(seed, 1, n_pages, kv_heads, page, d, nan_pages=True)
    values = random_pool(seed + 1, 1, n_pages, kv_heads, page, d)[0][1]
    table = np.full((len(seqs), max(map(len, seqs)) + 1), -1, np.int32)
    ids = iter(rng.permutation(n_pages))
    for b, pages in enumerate(seqs):
        for p, (ev, score) in enumerate(pages):
            i = table[b, p] = int(next(ids))
            k = np.zeros((kv_heads, page, d))
            k[..., 1:] = rng.standard_normal((kv_heads, page, d - 1)) * share
            k[..., 0] = np.broadcast_to(np.asarray(score, np.float64), (page,))
            codes[0][0, i] = torch.from_numpy(P.e4m3_code(P.e4m3_round(k)))
            codes[1][0, i] = values[0, i]
            exps[0][0, i], exps[1][0, i] = 0, ev
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    return cache_of(codes, exps), pool, table


def query(seed, rows, heads, d, signs):
    """Rows whose first channel is 1 or -1 (signs, repeated over rows and
    heads), the others small."""
    x = np.random.default_rng(seed).standard_normal((rows, heads, d)) * 0.02
    x[..., 0] = np.resize(np.asarray(signs, np.float64), rows * heads).reshape(rows, heads)
    return torch.from_numpy(x).float().bfloat16()


def dropped(pool, q, table, lens, counts, causal, window):
    """What the FP16 weights may leave out, per row: a weight of key j is
    p_j 2^ev_j in units in which the row's largest is 2^9 or more, rounded to a
    step of 2^-24 at least: 2^-25 off, 2^-34 of the largest, times a code of
    448 at most, for each key."""
    rows, hq, d = q.shape
    out, at = np.zeros((rows, hq)), 0
    for b, (length, n) in enumerate(zip(lens, counts)):
        k = pool.rows(0, table[b], length)
        ev = np.repeat(pool.exp[1][table[b][:-(-length // pool.page)]], pool.page, 0)[:length]   # [keys, heads]
        j = np.arange(length)
        for i in range(n):
            t = length - n + i
            see = (j <= t if causal else j >= 0) & (j > t - window if window else j >= 0)
            for h in range(hq):
                g = h // (hq // k.shape[0])
                s = k[g][see] @ q[at + i, h]          # in binades
                if len(s):
                    p = np.exp2(s - s.max())
                    out[at + i, h] = (p / p.sum() * 2.0 ** ev[see, g]).max() * 448 * 2.0 ** -34 * len(s)
        at += n
    return out


def check(got, pool, q, table, lens, counts, causal=True, window=0, rows=None):
    """Against the 64-bit oracle.  To the tolerances of the other tests come
    the left-out weights and the exponent's argument, which spans the scales'
    120 binades besides the weights' own 32 at most and is rounded in fp32:
    152 2^-24 binades, on the weight and on its sum."""
    x = q.double().numpy()
    ref = P.attention(pool, x, table, lens, counts, LN2, causal, window)
    out, lse, bound, serr, qerr = ref
    d, n_keys = q.shape[2], max(lens)
    tol_o, tol_l = tolerances(out, lse, bound, serr, qerr, d, n_keys)
    arg = 152 * 2.0 ** -24 * LN2
    tol_o = tol_o + 2 * arg * bound + dropped(pool, x, table, lens, counts, causal, window)[..., None]
    tol_l = tol_l + arg
    o, z = (g.float().cpu().numpy().astype(np.float64) for g in got)
    if rows is not None:
        o, z = o[rows], z[rows]
    empty = ~np.isfinite(lse)
    assert np.array_equal(z == -np.inf, empty) and (o[empty] == 0).all()
    assert np.isfinite(o).all()
    off = np.abs(o - out) / np.maximum(tol_o, 1e-300)
    assert off.max() <= 1, ("out", float(off.max()), int((off > 1).sum()))
    far = np.abs(np.where(empty, 0, z) - np.where(empty, 0, lse)) / tol_l
    assert far.max() <= 1, ("lse", float(far.max()))


def attend(cache, q, table, lens, counts, causal=True, window=0):
    got = kvq.paged_attention(cache, q.cuda(), dev(table), dev(lens), offsets_of(counts), max_q=max(counts), scale=LN2,
                              causal=causal, window=window, with_lse=True)
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_OK
    return got


ROWS = [(128, 1, 1, 1), (64, 3, 1, 1), (128, 3, 4, 1), (64, 4, 2, 2), (64, 40, 1, 1), (128, 20, 2, 1), (128, 300, 1, 1),
        (64, 150, 4, 2)]     # d, query rows, q heads, cache heads


@pytest.mark.parametrize("d,n,hq,hkv", ROWS)
@pytest.mark.parametrize("span", [20, 36, 45, 61, 100, 120])
def test_weight_on_the_page_of_small_scale(d, n, hq, hkv, span):
    """Two pages, scales `span` binades apart, the small one favoured by more
    or by less than that (or, in rows of the other sign, the large one), in
    either order."""
    top = span // 2
    for gap in (span + 20, span // 2, 6):
        for order in (1, -1):
            pages = [(top, 0.0), (top - span, float(gap))][::order]
            cache, pool, table = build(span + gap, 16, d, hkv, [pages])
            q = query(3, n, hq, d, [1, 1, -1])
            got = attend(cache, q, table, [32], [n], causal=False)
            check(got, pool, q, table, [32], [n], causal=False)


@pytest.mark.parametrize("d,n,hq,hkv", [(128, 2, 1, 1), (64, 4, 3, 1), (128, 12, 1, 1), (64, 40, 1, 1), (128, 20, 6, 1),
                                        (64, 300, 1, 1), (128, 150, 4, 2)])
@pytest.mark.parametrize("span", [20, 36, 61, 120])
def test_large_page_that_a_row_does_not_see(d, n, hq, hkv, span):
    """The page of large scale lies behind the causal limit of the earlier
    rows; then, under a window, before the first key of the later ones."""
    page = 16
    small = -(-(n + 20) // page)
    top = span // 2
    pages = [(top - span, 1.5)] * small + [(top, 0.0)]
    length = small * page + 1              # the last row alone sees the large page
    cache, pool, table = build(span + n, page, d, hkv, [pages])
    q = query(4, n, hq, d, [1, -1, 1])
    check(attend(cache, q, table, [length], [n]), pool, q, table, [length], [n])
    pages = [(top, 0.0)] + [(top - span, 1.5)] * (small + 1)
    length = (small + 2) * page
    window = length - n + 1 - (page - 1)   # the first row's window begins at the large page's last key
    cache, pool, table = build(span + n + 1, page, d, hkv, [pages])
    check(attend(cache, q, table, [length], [n], window=window), pool, q, table, [length], [n], window=window)


@pytest.mark.parametrize("d,n,hq,hkv", [(128, 1, 2, 1), (64, 5, 3, 1), (64, 40, 1, 1), (128, 120, 1, 1), (128, 140, 2, 1),
                                        (64, 300, 1, 1)])
@pytest.mark.parametrize("span,low", [(19, -30), (23, -60), (30, -60), (36, -60), (61, -90), (120, -180)])
def test_large_page_met_on_the_way(d, n, hq, hkv, span, low):
    """Ordinary pages, then one of a large scale and no weight in some later
    tile of 128 keys, then ordinary pages again (and their mirror image, rows
    of the other sign: the large page takes everything)."""
    page, top = 16, span // 2
    for at in (0, 9, 30, 47):
        pages = [(top - span, float(i % 3) / 2) for i in range(48)]
        pages[at] = (top, float(low))
        cache, pool, table = build(span + at, page, d, hkv, [pages])
        q = query(5, n, hq, d, [1, 1, 1, -1])
        length = 48 * page - 3
        check(attend(cache, q, table, [length], [n], causal=False), pool, q, table, [length], [n], causal=False)


@pytest.mark.parametrize("d,n,hq,batch", [(64, 1, 2, 1), (128, 3, 4, 1), (64, 24, 1, 1), (64, 1, 8, 310), (128, 2, 8, 310),
                                          (64, 24, 1, 310), (128, 60, 2, 310), (64, 130, 1, 310), (128, 200, 2, 310)])
@pytest.mark.parametrize("first", [True, False])
def test_many_keys_that_count_only_in_the_sum(d, n, hq, batch, first):
    """One key of the largest scale against 1000 or 8000 of the smallest, 16
    binades lower each: 2^-6 or an eighth of the softmax's sum and nothing in
    the output.  Many sequences (on the same pages) keep one sequence's keys in
    one CTA."""
    page, small = 64, 125 if batch == 1 else 15
    one = tuple([0.0] + [-200.0] * (page - 1))
    pages = [(-60, -16.0)] * small
    pages.insert(0 if first else small, (60, one))
    cache, pool, table = build(7, page, d, 1, [pages], share=0.01)
    q = query(6, n * batch, hq, d, [1])
    lens = [(small + 1) * page] * batch
    got = attend(cache, q, np.repeat(table, batch, 0), lens, [n] * batch, causal=False)
    check(got, pool, q[:n], table, lens[:1], [n], causal=False, rows=slice(0, n))


@pytest.mark.parametrize("d,page,hq,hkv,batch,n", [
    (128, 32, 16, 8, 50, 1), (64, 16, 16, 8, 60, 2), (128, 64, 32, 8, 40, 4),    # equal runs of the line
    (64, 32, 8, 4, 40, 1),                                                       # a CTA an item
    (128, 32, 2, 1, 3, 1), (64, 16, 4, 2, 2, 3),                                 # clusters
    (64, 32, 4, 1, 1, 9), (128, 64, 4, 2, 2, 40)])                               # tensor cores, keys in ranges
def test_scales_of_every_page_their_own(d, page, hq, hkv, batch, n):
    """Exponents all over the range, scores too, the keys divided among warps,
    CTAs and ranges in every way there is."""
    rng = np.random.default_rng(d + batch)
    seqs, lens = [], []
    for b in range(batch):
        length = int(rng.integers(900, 2500)) if batch < 8 else int(rng.integers(1, 700))
        lens.append(max(length, n))
        seqs.append([(int(rng.integers(-60, 61)), float(rng.integers(-70, 71))) for _ in range(-(-lens[-1] // page))])
    cache, pool, table = build(batch + n, page, d, hkv, seqs)
    counts = [n] * batch
    q = query(8, n * batch, hq, d, [1, -1, -1, 1, 1])
    got = attend(cache, q, table, lens, counts)
    for b in {0, 1, batch // 2, batch - 1} & set(range(batch)):
        rows = slice(b * n, (b + 1) * n)
        check(got, pool, q[rows], table[b:b + 1], lens[b:b + 1], [n], rows=rows)
    again = attend(cache, q, table, lens, counts)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("d,n,hq,hkv", ROWS)
@pytest.mark.parametrize("e", [0, 18, 22, 40, 60])
@pytest.mark.parametrize("span", [0, 30, 120])
def test_keys_of_any_scale(d, n, hq, hkv, e, span):
    """Key scales up to the largest, scores up to 2^69 binades: one key takes
    everything, by half of the scores' size or more, and the output is its
    value (in 16 bits); the logarithm is its score."""
    page, length = 16, 400
    rng = np.random.default_rng(e + n)
    n_pages = length // page
    codes, exps = random_pool(e + d, 1, n_pages, hkv, page, d)
    k0 = rng.uniform(-200, 200, (n_pages, hkv, page))
    best, worst = rng.permutation(length)[:2]
    k0[best // page, :, best % page], k0[worst // page, :, worst % page] = 448.0, -448.0
    k = np.zeros((n_pages, hkv, page, d))
    k[..., 0] = k0
    codes[0][0] = torch.from_numpy(P.e4m3_code(P.e4m3_round(k)))
    exps[0][:] = e
    exps[1][:] = rng.integers(-(span // 2), span // 2 + 1, exps[1].shape)
    cache = cache_of(codes, exps)
    q = query(9, n, hq, d, [1, -1, 1])
    table = np.arange(n_pages, dtype=np.int32)[None]
    scale = 0.3                                  # times log2 e: not a power of two
    got = kvq.paged_attention(cache, q.cuda(), dev(table), dev([length]), offsets_of([n]), max_q=n, scale=scale,
                              causal=False, with_lse=True)
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_OK
    values = P.Pool([c[0].numpy() for c in codes], [x[0] for x in exps]).rows(1, table[0], length)
    gap = scale * 248 * 2.0 ** e                 # from the winner's score to any other's, in nats, or more
    for h in range(hq):
        for i in range(n):
            v = values[h // (hq // hkv)]
            want = v[best if q[i, h, 0] > 0 else worst]
            # all others together: 400 e^-gap of at most 448 2^(span / 2)
            rest = 400 * math.exp(-min(gap, 700.0)) * 448 * 2.0 ** (span // 2)
            o = got[0][i, h].double().cpu().numpy()
            assert (np.abs(o - want) <= 2.0 ** -8 * np.abs(want) + rest).all(), (h, i)
            z, s = float(got[1][i, h]), scale * 448.0 * 2.0 ** e
            assert abs(z - s) <= s * 2.0 ** -20, (h, i, z, s)
