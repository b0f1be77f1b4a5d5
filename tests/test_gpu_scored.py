"""Attention over the paged cache with shaped scores (cap, distance bias) and
further masks (prefix, ranges) on the GPU, against the 64-bit oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from quantized_kv_cache_quantize_gb300 import kvq
from tests.paged_common import cache_of, check_attention, dev, make_table, offsets_of, random_pool, tolerances

pytestmark = pytest.mark.gpu


def clean():
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_OK


def rows_of(rng, rows, heads, d, spread=0.3, heat=1.0):
    x = rng.standard_normal((rows, heads, d)) * np.exp(rng.standard_normal((rows, heads, 1)) * spread) * heat
    return torch.from_numpy(x).float().bfloat16()


def pool_case(seed, lens, page, heads, d, **kw):
    rng = np.random.default_rng(seed)
    n_pages = sum(-(-n // page) for n in lens) + 2
    codes, exps = random_pool(seed, 1, n_pages, heads, page, d, **kw)
    return rng, codes, exps, make_table(rng, lens, page, n_pages)


def check(got, ref, d, n_keys, softcap, what=""):
    """check_attention's bounds with two more terms.
    - The shaping's own rounding, as a score's error.  cap (1 - 2 r), r = 1 / (1 +
      t) by one reciprocal of a pair's product: r is off by 2^-23 (the reciprocal)
      and 3 2^-24 (1 + t, the product, its share), 5 2^-23 of the cap as 2 r; t by
      2^-21 (the exponential 2^-22, its argument as much where the derivative
      counts), 2 2^-23 of the cap as 2 t / (1 + t)^2 is 1/2 at most; the sum
      2^-24: 2^-20 of the cap in all.  A bias: three roundings, 2^-22 of |score| +
      |bias|; log2 units and back, the same again.  It enters serr, which
      tolerances() takes times (d + 4) 2^-23.
    - Weights times V scales in FP16 are off by half a subnormal step, 2^-25,
      where the largest of the row stands at 2^9 or above: 2^-34 of that largest
      per key, times a code of 448 at most, whatever the channel's own sum is.
      (tolerances() has 2^-34 a key of the channel's sum p |v|, which is less
      where the keys that lead the row hold zeros in a channel: with hot scores,
      d = 128 and 333 and 90 keys, row 30 of head 3 has 1.1e-19 in channel 82, all
      of it from weights below 2^-60 of the largest; FP16 leaves 0.)"""
    out, lse, bound, serr, qerr, herr, top = ref
    extra = 2.0 ** -20 * softcap + 2.0 ** -21 * herr
    tol_o, tol_l = tolerances(out, lse, bound, serr + extra / ((d + 4) * 2.0 ** -23), qerr, d, n_keys)
    tol_o = tol_o + (n_keys * 448 * 2.0 ** -34 * top)[..., None]
    o, z = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    assert np.isfinite(o).all(), what
    empty = ~np.isfinite(lse)
    assert np.array_equal(z == -np.inf, empty), what
    assert (o[empty] == 0).all(), what
    over = np.abs(o - out) > tol_o
    assert not over.any(), (what, "out", int(over.sum()), float((np.abs(o - out) / np.maximum(tol_o, 1e-300)).max()))
    far = np.abs(np.where(empty, 0, z) - np.where(empty, 0, lse)) > tol_l
    assert not far.any(), (what, "lse", int(far.sum()), float(np.nanmax(np.abs(z - lse))))


def slopes_of(hq, rng=None):
    return np.array([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], np.float32)


def docs_of(rng, lens, counts, n_docs, empty=0.1):
    """The ranges of rows in documents at random cuts; some rows see nothing."""
    out = []
    for length, n in zip(lens, counts):
        cuts = np.unique(np.concatenate([[0], rng.integers(0, max(length, 1), n_docs - 1), [max(length, 1)]]))
        for t in range(length - n, length):
            k = int(np.searchsorted(cuts, max(t, 0), side="right")) - 1
            out.append((5, 5) if rng.random() < empty else (int(cuts[k]), int(cuts[min(k + 1, len(cuts) - 1)])))
    return np.array(out, np.int64).reshape(-1, 2)


CASES = [  # d, page, q heads, cache heads, lengths, query rows, causal, window, softcap, slopes, prefix, documents
    (128, 16, 1, 1, [1], [1], True, 0, 10.0, True, False, 0),
    (64, 16, 3, 3, [5, 16, 17], [1, 1, 1], True, 0, 5.0, False, False, 0),
    (128, 64, 8, 2, [300, 1, 64, 0, 65], [1, 1, 1, 1, 1], True, 0, 0.0, True, False, 0),
    (128, 32, 10, 2, [513, 100], [1, 1], False, 0, 3.0, True, False, 4),
    (64, 128, 16, 1, [1000, 3], [1, 1], True, 100, 20.0, False, True, 0),
    (128, 16, 14, 2, [700, 30, 250], [1, 1, 1], True, 33, 0.0, True, False, 3),
    (128, 64, 32, 1, [200], [1], True, 0, 2.0, True, False, 0),
    (64, 32, 8, 4, [90, 40, 33], [4, 2, 7], True, 0, 0.0, False, True, 3),
    (128, 64, 6, 2, [500, 3, 130], [5, 5, 0], True, 64, 4.0, True, True, 2),      # rows before the first key
    (128, 16, 4, 4, [130], [3], False, 0, 0.0, True, False, 0),
    (128, 64, 4, 2, [300, 129], [300, 70], True, 0, 4.0, False, True, 0),
    (64, 64, 4, 4, [260], [129], False, 0, 1.0, True, False, 5),
    (128, 32, 5, 1, [400, 77, 20], [90, 77, 33], True, 50, 0.0, True, False, 4),
    (128, 128, 2, 2, [257, 1], [128, 1], False, 0, 0.0, True, False, 0),
    (64, 16, 7, 1, [333], [61], True, 17, 6.0, True, True, 3),
    (128, 16, 2, 1, [40], [150], True, 0, 3.0, True, True, 0),                     # more rows than keys
    (64, 128, 24, 8, [150, 300], [1, 65], False, 90, 0.0, False, False, 7),
    (128, 64, 3, 1, [640], [1], True, 1, 2.0, True, False, 0),
    (64, 32, 8, 1, [1500, 1100], [5, 5], True, 0, 7.0, True, True, 2),             # one row tile, many key tiles
    (128, 64, 2, 1, [1300], [50], False, 1100, 0.0, True, False, 0),
    (128, 128, 2, 1, [900], [140], True, 0, 5.0, False, True, 6),
    (64, 64, 1, 1, [700], [300], True, 0, 0.0, False, False, 40),                  # 256 tokens in one tile, short documents
    (128, 32, 1, 1, [515], [515], True, 0, 0.0, True, False, 0),
    (64, 16, 2, 2, [2100], [200], True, 0, 9.0, True, False, 2),
]


def run_case(d, page, hq, hkv, lens, counts, causal, window, softcap, slopes, prefix, docs, seed=0, heat=1.0, scale=None):
    rng, codes, exps, table = pool_case(d + sum(lens) + seed, lens, page, hkv, d, e_lo=-9, e_hi=-5)
    q = rows_of(rng, sum(counts), hq, d, heat=heat)
    scale = 1 / np.sqrt(d) if scale is None else scale
    # whatever the last pages hold behind the lengths must not matter
    codes = [c.clone() for c in codes]
    for b, n in enumerate(lens):
        if n % page:
            for c in codes:
                c[0, table[b][n // page], :, n % page:] = 0x7F
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    kw = dict(slopes=slopes_of(hq) if slopes else None,
              prefix=np.array([int(n * rng.random()) for n in lens]) if prefix else None,
              ranges=docs_of(rng, lens, counts, docs) if docs else None)
    ref = P.attention_scored(pool, q.double().numpy(), table, lens, counts, scale, causal, window, softcap, **kw)
    kw = {k: None if v is None else dev(v, torch.float32 if k == "slopes" else torch.int32) for k, v in kw.items()}
    cache = cache_of(codes, exps)
    one = all(n == 1 for n in counts)
    for off in ([offsets_of(counts)] + ([None] if one else [])):
        got = kvq.paged_attention(cache, q.cuda(), dev(table), dev(lens), off, causal=causal, window=window, scale=scale,
                                  with_lse=True, max_q=max(counts), softcap=softcap, **kw)
        clean()
        check(got, ref, d, max(lens), softcap, str((lens, counts)))


@pytest.mark.parametrize("d,page,hq,hkv,lens,counts,causal,window,softcap,slopes,prefix,docs", CASES)
def test_scored(d, page, hq, hkv, lens, counts, causal, window, softcap, slopes, prefix, docs):
    run_case(d, page, hq, hkv, lens, counts, causal, window, softcap, slopes, prefix, docs)


@pytest.mark.parametrize("d,hq,hkv,rows", [(128, 4, 4, 1), (64, 6, 3, 2), (128, 12, 4, 3)])
@pytest.mark.parametrize("softcap,slopes,prefix,docs", [(5.0, True, True, 4), (0.0, False, False, 3), (8.0, False, False, 0)])
def test_many_short_sequences(d, hq, hkv, rows, softcap, slopes, prefix, docs):
    """More (sequence, head) pairs than two for every SM: the line of all keys."""
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(0, 150, 110)]
    lens[3], lens[50] = 700, 0
    run_case(d, 32, hq, hkv, lens, [min(rows, max(1, n)) for n in lens], True, 60 if docs else 0, softcap, slopes, prefix, docs, seed=1)


@pytest.mark.parametrize("d,page,rows", [(128, 128, 1), (64, 16, 2)])
@pytest.mark.parametrize("softcap,slopes,prefix,docs", [(5.0, True, False, 0), (0.0, True, False, 5)])
def test_one_long_sequence(d, page, rows, softcap, slopes, prefix, docs):
    """Few pairs: clusters of CTAs share the keys of one."""
    run_case(d, page, 4, 2, [9000], [rows], True, 0, softcap, slopes, prefix, docs, seed=2)


@pytest.mark.parametrize("softcap", [2.0 ** -20, 1e-3, 0.7, 50.0, 1000.0, 2.0 ** 20])
@pytest.mark.parametrize("hq,counts", [(2, [1, 3]), (8, [2, 2]), (4, [70, 9]), (2, [200, 90])])
def test_caps_of_every_size(softcap, hq, counts):
    """From scores that all lie at the cap to scores that do not feel it."""
    run_case(128, 32, hq, 1, [333, 90], counts, True, 0, softcap, False, False, 0, heat=8.0)


@pytest.mark.parametrize("counts", [[1, 1], [4, 1], [100, 20], [260, 30]])
def test_scores_of_some_hundreds(counts):
    """Hot rows: the cap decides which keys share a row."""
    run_case(128, 16, 4, 2, [300, 64], counts, True, 0, 30.0, True, False, 0, heat=20.0, scale=1.0)
    run_case(64, 64, 4, 4, [300, 64], counts, True, 0, 300.0, False, False, 0, heat=20.0, scale=1.0)


@pytest.mark.parametrize("slope", [0.0, 4.0, 300.0, -0.02])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,counts", [(3, [1, 2]), (2, [8, 3]), (3, [60, 120])])
def test_slopes_of_every_size(slope, causal, hq, counts):
    """No bias, one that leaves a row its nearest keys, one that leaves it one,
    one that grows with the distance."""
    d, lens, page = 64, [700, 150], 32
    rng, codes, exps, table = pool_case(3, lens, page, 1, d, e_lo=-9, e_hi=-6)
    q = rows_of(rng, sum(counts), hq, d)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    s = np.full(hq, slope, np.float32)
    s[0] = 0.01
    ref = P.attention_scored(pool, q.double().numpy(), table, lens, counts, 0.125, causal, 0, slopes=s)
    got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of(counts), causal=causal,
                              with_lse=True, max_q=max(counts), slopes=dev(s, torch.float32))
    clean()
    check(got, ref, d, 700, 0.0)


@pytest.mark.parametrize("hq,counts", [(2, [1, 1, 1]), (4, [3, 4, 2]), (2, [90, 40, 130])])
def test_any_number_is_a_prefix_or_a_bound(hq, counts):
    d, lens, page = 64, [300, 41, 130], 16
    rng, codes, exps, table = pool_case(4, lens, page, 2, d, e_lo=-9, e_hi=-6)
    rows, top = sum(counts), 2 ** 31 - 1
    q = rows_of(rng, rows, hq, d)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ends = np.array([-top - 1, -7, 0, 1, 20, 37, 300, 1000, top])
    ranges = np.stack([rng.choice(ends, rows), rng.choice(ends, rows)], 1)
    for prefix in ([-5, top, -top - 1], [1000, 0, 57]):
        for causal in (True, False):
            ref = P.attention_scored(pool, q.double().numpy(), table, lens, counts, 0.1, causal, 0, prefix=prefix, ranges=ranges)
            got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of(counts), scale=0.1,
                                      causal=causal, with_lse=True, max_q=max(counts), prefix=dev(prefix), ranges=dev(ranges))
            clean()
            check(got, ref, d, 300, 0.0)
    ref = P.attention_scored(pool, q.double().numpy(), table, lens, counts, 0.1, True, 0, ranges=np.zeros((rows, 2), int))
    assert not np.isfinite(ref[1]).any()
    got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of(counts), scale=0.1,
                              with_lse=True, max_q=max(counts), ranges=torch.zeros(rows, 2, dtype=torch.int32, device="cuda"),
                              softcap=4.0)
    clean()
    check(got, ref, d, 300, 0.0)


@pytest.mark.parametrize("d,page,hq,rows", [(128, 16, 2, 1), (64, 32, 4, 2), (128, 64, 8, 2), (64, 16, 2, 40), (128, 128, 2, 70),
                                            (64, 64, 1, 300)])
@pytest.mark.parametrize("softcap", [0.0, 8.0])
def test_what_no_row_sees_does_not_matter(d, page, hq, rows, softcap):
    """NaN codes between the rows' ranges, before the first and behind the last,
    and no page at all where a whole one lies outside them."""
    lens = [600, 500]
    rng, codes, exps, table = pool_case(7, lens, page, 1, d, e_lo=-9, e_hi=-6)
    counts = [rows, rows]
    q = rows_of(rng, 2 * rows, hq, d)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ranges = np.zeros((2 * rows, 2), int)
    for r in range(2 * rows):
        ranges[r] = [(150, 163), (260, 261), (200, 240), (30, 30)][r % 4]
    ref = P.attention_scored(pool, q.double().numpy(), table, lens, counts, 0.1, False, 0, softcap, ranges=ranges)
    codes = [c.clone() for c in codes]
    for b in range(2):
        mine = [tuple(x) for x in ranges[b * rows:(b + 1) * rows]]
        for j in range(lens[b]):
            if not any(lo <= j < hi for lo, hi in mine):
                for c in codes:
                    c[0, table[b][j // page], :, j % page] = 0x7F
        lo, hi = min([m[0] for m in mine if m[1] > m[0]] or [0]), max([m[1] for m in mine if m[1] > m[0]] or [0])
        table[b, :lo // page] = -1
        table[b, -(-hi // page):] = 1 << 30
    got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of(counts), scale=0.1,
                              causal=False, with_lse=True, max_q=rows, softcap=softcap, ranges=dev(ranges))
    clean()
    check(got, ref, d, 600, softcap)


@pytest.mark.parametrize("hq,rows", [(2, 1), (4, 4), (2, 70), (2, 300)])
def test_far_pages_by_scale(hq, rows):
    """Value pages 100 binades apart beside a cap and a bias: which page decides
    the output differs from which decides the sum."""
    d, page, lens = 64, 16, [300]
    for lo_hi in ((-50, 50), (-5, 0)):
        rng, codes, exps, table = pool_case(9, lens, page, 1, d, e_lo=-9, e_hi=-6)
        exps[1][0] = rng.integers(lo_hi[0], lo_hi[1] + 1, exps[1][0].shape)
        q = rows_of(rng, rows, hq, d)
        pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
        s = np.array([0.5, 0.02, 0.1, 0.0], np.float32)[:hq]
        for softcap, slopes in ((6.0, None), (0.0, s), (6.0, s)):
            ref = P.attention_scored(pool, q.double().numpy(), table, lens, [rows], 0.1, True, 0, softcap, slopes)
            got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of([rows]), scale=0.1,
                                      with_lse=True, max_q=rows, softcap=softcap,
                                      slopes=None if slopes is None else dev(slopes, torch.float32))
            clean()
            check(got, ref, d, 300, softcap)


@pytest.mark.parametrize("rows", [1, 5, 200])
def test_not_finite_rows_and_seen_keys(rows):
    """A row with an infinity is NaN and nobody else; a key with a NaN is in the
    results of the rows that attend to it and in no others'."""
    d, page, lens = 64, 16, [400]
    rng, codes, exps, table = pool_case(2, lens, page, 1, d, e_lo=-9, e_hi=-6)
    q = rows_of(rng, rows, 2, d)
    q[rows // 2, 1, 3] = float("inf")
    ranges = np.tile([[10, 20]], (rows, 1))
    ranges[0] = [100, 140]
    codes = [c.clone() for c in codes]
    codes[0][0, table[0][7], 0, 2, 5] = 0x7F                                  # key 114
    got, lse = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of([rows]), causal=False,
                                   with_lse=True, max_q=rows, softcap=9.0, ranges=dev(ranges))
    clean()
    want = torch.zeros(rows, 2, dtype=torch.bool)
    want[rows // 2, 1] = want[0] = True
    nan = torch.isnan(got.float()).cpu()
    assert torch.equal(nan.all(-1), want) and torch.equal(nan.any(-1), want) and torch.equal(torch.isnan(lse).cpu(), want)


@pytest.mark.parametrize("rows", [2, 70, 300])
@pytest.mark.parametrize("softcap,slope", [(0.0, 0.0), (5.0, 0.0), (0.0, 0.01), (5.0, 0.01)])
@pytest.mark.parametrize("nan", [False, True])
def test_rows_that_see_nothing_beside_rows_that_see_all(rows, softcap, slope, nan):
    """Padding rows in the middle of others, whole tiles around them: zero and
    -infinity, also where a value that the others attend to is a NaN."""
    d, page, lens = 128, 64, [640]
    rng, codes, exps, table = pool_case(17, lens, page, 2, d, e_lo=-9, e_hi=-6)
    q = rows_of(rng, rows, 2, d)
    ranges = np.tile([[0, 640]], (rows, 1))
    ranges[1::3] = [[0, 0]]
    if nan:
        codes = [c.clone() for c in codes]
        codes[1][0, table[0][2], :, 5, 7] = 0x7F
    s = dev(np.full(2, slope), torch.float32)
    out, lse = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of([rows]), scale=0.1,
                                   causal=False, with_lse=True, max_q=rows, softcap=softcap, slopes=s, ranges=dev(ranges))
    clean()
    assert (out[1::3] == 0).all() and (lse[1::3] == -np.inf).all()
    assert torch.isnan(out[0::3, :, 7]).all() if nan else torch.isfinite(out[0::3]).all()
    if not nan:
        pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
        ref = P.attention_scored(pool, q.double().numpy(), table, lens, [rows], 0.1, False, 0, softcap, np.full(2, slope), ranges=ranges)
        check((out, lse), ref, d, 640, softcap)


def test_rows_that_see_nothing_in_many_sequences():
    """The same in the line of all keys, single tokens and pairs of 160 sequences."""
    d, page, batch = 64, 32, 160
    lens = [64] * batch
    rng, codes, exps, table = pool_case(18, lens, page, 2, d, e_lo=-9, e_hi=-6)
    q = rows_of(rng, 2 * batch, 2, d)
    ranges = np.tile([[0, 64], [7, 7]], (batch, 1))
    codes = [c.clone() for c in codes]
    codes[1][0, table[:, 0], :, 5, 7] = 0x7F
    out, lse = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of([2] * batch), scale=0.1,
                                   causal=False, with_lse=True, max_q=2, softcap=5.0, ranges=dev(ranges))
    clean()
    assert (out[1::2] == 0).all() and (lse[1::2] == -np.inf).all() and torch.isnan(out[0::2, :, 7]).all()


@pytest.mark.parametrize("rows", [1, 5, 70, 300])
@pytest.mark.parametrize("power", [12, 30])
def test_scores_beyond_every_bias(rows, power):
    """Scores of 2^12 and 2^30 beside a bias: two equal keys, tiles apart, share
    the row, whatever the rounding of a base that large; the others weigh nothing."""
    d, page, n = 64, 64, 900
    lens = [n]
    rng, codes, exps, table = pool_case(14, lens, page, 1, d, e_lo=0, e_hi=0)
    k = np.zeros((exps[0].shape[1], 1, page, d))
    k[..., 0] = rng.integers(1, 8, k.shape[:-1]) / 8.0
    best = (65, 700)
    for j in best:
        k[table[0][j // page], 0, j % page, 0] = 2.0
    codes[0][0] = torch.from_numpy(P.e4m3_code(P.e4m3_round(k)))
    q = torch.zeros(rows, 2, d, dtype=torch.bfloat16)
    q[..., 0] = 2.0 ** power
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    s = np.array([0.0, 2.0 ** -30], np.float32)
    ref = P.attention_scored(pool, q.double().numpy(), table, lens, [rows], 0.5, False, 0, slopes=s)
    got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of([rows]), scale=0.5,
                              causal=False, with_lse=True, max_q=rows, slopes=dev(s, torch.float32))
    clean()
    assert np.abs(ref[0][:, 0] - (pool.rows(1, table[0], n)[0][list(best)]).mean(0)).max() < 1e-12
    check(got, ref, d, n, 0.0)


@pytest.mark.parametrize("rows", [1, 5, 70, 300])
@pytest.mark.parametrize("heat", [1.0, 20.0])
def test_masked_neighbours_of_seen_keys(rows, heat):
    """NaN in every key that a row's range leaves out, right beside those that it
    sees, at odd and even places; scores below the cap and far beyond it."""
    d, page, lens = 64, 32, [500]
    rng, codes, exps, table = pool_case(12, lens, page, 2, d, e_lo=-9, e_hi=-6)
    q = rows_of(rng, rows, 2, d, heat=heat)
    ranges = np.tile([[101, 130]], (rows, 1))
    ranges[rows // 2:] = [[102, 131]]
    if rows == 1:
        ranges[0] = [101, 131]
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    codes = [c.clone() for c in codes]
    for j in list(range(101)) + list(range(131, 500)):
        for c in codes:
            c[0, table[0][j // page], :, j % page] = 0x7F
    codes[0][0, table[0][101 // page], :, 101 % page] = 0x7F                   # K alone: V is weighed by zero there
    for sl in (slice(0, rows // 2), slice(rows // 2, rows)):
        if rows == 1 or sl.start == 0:
            continue
        ref = P.attention_scored(pool, q.double().numpy(), table, lens, [rows], 0.2, False, 0, 6.0, ranges=ranges)
        got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of([rows]), scale=0.2,
                                  causal=False, with_lse=True, max_q=rows, softcap=6.0, ranges=dev(ranges))
        clean()
        check([g[sl] for g in got], [x[sl] for x in ref], d, 30, 6.0, str(sl))
        assert torch.isnan(got[1][:rows // 2]).all()                            # these see key 101


@pytest.mark.parametrize("hq,counts", [(4, [1, 1]), (4, [3, 2]), (4, [70, 5]), (2, [200, 90])])
def test_without_shapes_it_is_the_plain_call(hq, counts):
    """Shapes that change nothing: a prefix of no token, ranges over everything;
    the outputs are the plain call's within its tolerance."""
    d, lens, page = 128, [300, 140], 32
    rng, codes, exps, table = pool_case(6, lens, page, 2, d, e_lo=-9, e_hi=-6)
    q = rows_of(rng, sum(counts), hq, d)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ref = P.attention(pool, q.double().numpy(), table, lens, counts, 0.1, True, 70)
    all_keys = dev(np.tile([[0, 2 ** 31 - 1]], (sum(counts), 1)))
    for kw in (dict(prefix=dev([0, 0])), dict(ranges=all_keys), dict(slopes=torch.zeros(hq, device="cuda"))):
        got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of(counts), scale=0.1,
                                  window=70, with_lse=True, max_q=max(counts), **kw)
        clean()
        check_attention(got, ref, d, 300)


def test_refusals_on_the_device():
    cache = kvq.PagedCache.zeros(1, 4, 2, 16, 64)
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    table, lens = dev([[0], [1]]), dev([1, 1])
    for name, bad in (("slopes", torch.ones(2, device="cuda")), ("slopes", torch.ones(4, device="cuda").double()),
                      ("slopes", torch.ones(4)), ("slopes", torch.ones(8, device="cuda")[::2]),
                      ("prefix", dev([1])), ("prefix", dev([1, 1]).long()), ("ranges", dev([[0, 1]])),
                      ("ranges", dev([0, 1, 0, 1])), ("ranges", dev([[0, 0], [1, 1]]).T)):
        with pytest.raises(ValueError, match=name):
            kvq.paged_attention(cache, q, table, lens, **{name: bad})
    for cap in (-1.0, float("nan"), float("inf"), 2.0 ** -21, 2.0 ** 21, 1e-60):
        with pytest.raises(kvq.KVQError) as e:
            kvq.paged_attention(cache, q, table, lens, softcap=cap)
        assert e.value.status == kvq.KVQ_ERR_INVALID_ARG
    room = torch.zeros(5, dtype=torch.int32, device="cuda")
    with pytest.raises(kvq.KVQError) as e:
        kvq.paged_attention(cache, q, table, lens, ranges=room[1:].view(2, 2))
    assert e.value.status == kvq.KVQ_ERR_ALIGNMENT
    clean()


@pytest.mark.parametrize("counts", [[1, 1], [6, 40], [1, 300]])
def test_bad_pages_are_skipped_and_recorded(counts):
    d, page, lens = 128, 16, [100, 300]
    rng, codes, exps, table = pool_case(13, lens, page, 2, d, e_lo=-8, e_hi=-6)
    q = rows_of(rng, sum(counts), 2, d)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ref = P.attention_scored(pool, q.double().numpy(), table, lens, counts, 0.1, True, 0, 5.0, np.array([0.1, 0.2]))
    for wrong in (-1, codes[0].shape[1], 1 << 30):
        t = table.copy()
        t[0, 3] = wrong
        got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(t), dev(lens), offsets_of(counts), scale=0.1,
                                  with_lse=True, max_q=max(counts), softcap=5.0, slopes=dev([0.1, 0.2], torch.float32))
        torch.cuda.synchronize()
        assert kvq.last_device_status() == kvq.KVQ_ERR_PAGE
        r = counts[0]
        check([g[r:] for g in got], [x[r:] for x in ref], d, 300, 5.0)
        assert torch.isfinite(got[0]).all()


def test_rows_outside_the_offsets_are_left():
    rng, codes, exps, table = pool_case(5, [60], 16, 1, 64, e_lo=-8, e_hi=-6)
    for rows, hq in ((8, 2), (60, 2)):
        q = rows_of(rng, rows + 9, hq, 64).cuda()
        q[:4], q[4 + rows:] = float("nan"), float("nan")
        out = torch.full_like(q, 7.0)
        kvq.paged_attention(cache_of(codes, exps), q, dev(table), dev([60]), dev([4, 4 + rows]), max_q=rows, out=out,
                            softcap=3.0, ranges=dev(np.tile([[0, 60]], (rows + 9, 1))))
        clean()
        assert (out[:4] == 7).all() and (out[4 + rows:] == 7).all() and torch.isfinite(out[4:4 + rows]).all()


@pytest.mark.parametrize("hq,counts", [(4, [1, 1]), (4, [2, 3]), (2, [70, 300])])
def test_streams_and_graphs(hq, counts):
    """On a stream of its own and captured: a replay follows slopes, prefixes,
    ranges and lengths that changed; twice the same gives the same bits."""
    d, lens, page = 64, [2000, 310], 32
    rng, codes, exps, table = pool_case(6, lens, page, 2, d, e_lo=-9, e_hi=-6)
    q = rows_of(rng, sum(counts), hq, d).cuda()
    cache, t, n = cache_of(codes, exps), dev(table), dev(lens)
    off = offsets_of(counts)
    s, p = torch.full((hq,), 0.02, device="cuda"), dev([50, 7])
    r = dev(docs_of(rng, lens, counts, 3))

    def call(lens_, s_, p_, r_, **kw):
        return kvq.paged_attention(cache, q, t, lens_, off, max_q=max(counts), with_lse=True, softcap=5.0, slopes=s_,
                                   prefix=p_, ranges=r_, **kw)

    first, again = call(n, s, p, r), call(n, s, p, r)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = call(n, s, p, r, stream=side)
    side.synchronize()
    clean()
    for x, y, z in zip(first, again, other):
        assert torch.equal(x, y) and torch.equal(x, z)
    n0, s0, p0, r0 = n.clone(), s.clone(), p.clone(), r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(n0, s0, p0, r0)
    graph.replay()
    clean()
    assert all(torch.equal(a, b) for a, b in zip(out, first))
    n0.sub_(3)
    s0.fill_(0.3)
    p0.fill_(33)
    r0[:, 0] += 2
    graph.replay()
    clean()
    want = call(n - 3, s * 0 + 0.3, p * 0 + 33, r0)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_a_layer_as_it_is_used():
    """Rotated append, then capped attention with documents, prompt and single
    tokens after it, against the oracle over the same pages."""
    rng = np.random.default_rng(21)
    d, page, heads, hq = 128, 16, 2, 6
    f = kvq.rope_frequencies(64)
    rot = kvq.RopeTable.build(400, f)
    cs = rot.cos_sin.cpu().numpy()
    cache = kvq.PagedCache.zeros(1, 20, heads, page, d)
    pool = P.Pool([np.zeros((20, heads, page, d), np.uint8)] * 2, [np.zeros((20, heads), int)] * 2)
    lens = [0, 0]
    table = make_table(rng, [150, 90], page, 20)
    for step, counts in enumerate(([140, 77], [1, 1], [1, 1], [4, 2])):
        lens = [a + b for a, b in zip(lens, counts)]
        rows = sum(counts)
        q, k, v = (rows_of(rng, rows, h, d) for h in (hq, heads, heads))
        pos = np.concatenate([np.arange(n - c, n) for n, c in zip(lens, counts)])[:, None]
        off = None if step in (1, 2) else offsets_of(counts)
        turned = kvq.pages_append_rope(cache, rot, k.cuda(), v.cuda(), dev(table), dev(lens), off, q=q.cuda())
        ranges = np.concatenate([[((0, 60) if t < 60 else (60, 1000)) for t in range(n - c, n)] for n, c in zip(lens, counts)])
        got = kvq.paged_attention(cache, turned, dev(table), dev(lens), off, max_q=max(counts), with_lse=True,
                                  softcap=15.0, ranges=dev(ranges))
        clean()
        P.append(pool, P.rope_steps(k.float().numpy(), cs, pos, [0] * 64, False), v.double().numpy(), table, lens, counts)
        qt = torch.from_numpy(P.rope_steps(q.float().numpy(), cs, pos, [0] * 64, False)).bfloat16()
        ref = P.attention_scored(pool, qt.double().numpy(), table, lens, counts, d ** -0.5, True, 0, 15.0, ranges=ranges)
        check(got, ref, d, max(lens), 15.0, what=str(step))


@pytest.mark.parametrize("hq,rows", [(4, 1), (2, 70)])
def test_calls_at_once(hq, rows):
    """Two calls under way on two streams, and two captured graphs replayed on
    two streams: nothing they share."""
    d, page, lens = 64, 32, [9000, 8000, 8500] if rows == 1 else [4000, 3000, 3500]
    rng, codes, exps, table = pool_case(16, lens, page, 2, d, e_lo=-9, e_hi=-6)
    cache, t, n, off = cache_of(codes, exps), dev(table), dev(lens), offsets_of([rows] * 3)
    qs = [rows_of(rng, 3 * rows, hq, d).cuda() for _ in range(2)]
    kws = [dict(softcap=4.0, ranges=dev(docs_of(rng, lens, [rows] * 3, 4))), dict(slopes=torch.full((hq,), 0.01, device="cuda"), prefix=dev([9, 8, 7]))]

    def call(i, **kw):
        return kvq.paged_attention(cache, qs[i], t, n, off, max_q=rows, with_lse=True, **kws[i], **kw)

    want = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [call(i, stream=s) for i, s in enumerate(streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, w in zip(got, want) for x, y in zip(g, w))
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(i))
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, w in zip(outs, want) for x, y in zip(g, w))
    clean()
