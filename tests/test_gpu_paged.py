"""The paged 8-bit cache on the GPU against its 64-bit oracle: codes, scales,
tables and counts bit for bit, attention within derived bounds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from quantized_kv_cache_quantize_gb300 import kvq
from tests.paged_common import (cache_of, check_attention, codes_of, dev, exps_of, make_table, offsets_of, random_pool)

pytestmark = pytest.mark.gpu


def clean():
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_OK


def rows_of(rng, rows, heads, d, spread=1.0):
    x = rng.standard_normal((rows, heads, d)) * np.exp(rng.standard_normal((rows, heads, 1)) * spread)
    return torch.from_numpy(x).float().bfloat16()


# ---- append ----

APPENDS = [  # d, page, heads, lengths after, new rows
    (128, 16, 2, [1], [1]),
    (64, 16, 1, [16, 17, 31], [1, 1, 1]),
    (128, 64, 3, [200, 1, 64, 65, 0], [200, 1, 64, 1, 0]),
    (64, 128, 2, [129, 300, 5], [2, 171, 0]),
    (128, 32, 5, [100, 33, 32, 7, 64], [68, 33, 1, 7, 31]),
    (64, 32, 4, [40] * 9, [1] * 9),
    (128, 128, 1, [1000], [873]),
    (64, 64, 8, [63, 130], [1, 67]),
]


@pytest.mark.parametrize("d,page,heads,lens,counts", APPENDS)
@pytest.mark.parametrize("strided", [False, True])
def test_append(d, page, heads, lens, counts, strided):
    rng = np.random.default_rng(sum(lens) + d + page)
    n_pages = sum(-(-n // page) for n in lens) + 2
    codes, exps = random_pool(3, 1, n_pages, heads, page, d, e_lo=-12, e_hi=-5)
    cache = cache_of(codes, exps)
    table = make_table(rng, lens, page, n_pages)
    rows = sum(counts)
    k, v = rows_of(rng, rows, heads, d), rows_of(rng, rows, heads, d, 0.3)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    P.append(pool, k.double().numpy(), v.double().numpy(), table, lens, counts)
    if strided:   # heads before rows, and every other row of a wider tensor
        kk = k.transpose(0, 1).contiguous().cuda().transpose(0, 1)
        vv = torch.zeros(2 * rows, heads + 1, d, dtype=torch.bfloat16)
        vv[::2, 1:] = v
        vv = vv.cuda()[::2, 1:]
    else:
        kk, vv = k.cuda(), v.cuda()
    one = all(n == 1 for n in counts)
    wide = torch.full((len(lens), table.shape[1] + 3), 7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = dev(table)
    for off in ([offsets_of(counts)] + ([None] if one else [])):
        cache = cache_of(codes, exps)
        kvq.pages_append(cache, kk, vv, wide[:, :table.shape[1]], dev(lens), off)
        clean()
        for kv, (c, s) in enumerate(((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale))):
            assert np.array_equal(exps_of(s)[0], pool.exp[kv])
            got = codes_of(c)[0]
            assert np.array_equal(P.VALUES[got], pool.val[kv])
            # pages no sequence writes keep their bytes
            written = {table[b][p] for b in range(len(lens)) for p in range(-(-lens[b] // page))
                       if (p + 1) * page > lens[b] - counts[b]}
            for i in set(range(n_pages)) - written:
                assert np.array_equal(got[i], codes[kv][0, i].numpy())


def test_append_layers_and_offsets_behind_the_last_sequence():
    """Only the named layer changes, and rows behind offsets[batch] are not read."""
    rng = np.random.default_rng(0)
    codes, exps = random_pool(1, 3, 6, 2, 16, 64)
    cache = cache_of(codes, exps)
    k = rows_of(rng, 20, 2, 64)
    k[10:] = float("nan")
    table = make_table(rng, [30], 16, 6)
    kvq.pages_append(cache, k.cuda(), k.cuda(), dev(table), dev([30]), dev([0, 10]), layer=1)
    clean()
    pool = P.Pool([c[1].numpy() for c in codes], [e[1] for e in exps])
    P.append(pool, k[:10].double().numpy(), k[:10].double().numpy(), table, [30], [10])
    for kv, c in enumerate((cache.k_codes, cache.v_codes)):
        got = codes_of(c)
        assert np.array_equal(got[0], codes[kv][0].numpy()) and np.array_equal(got[2], codes[kv][2].numpy())
        assert np.array_equal(P.VALUES[got[1]], pool.val[kv])


@pytest.mark.parametrize("value,e", [(0.0, -60), (1e-30, -60), (448.0, 0), (450.0, 1), (2.0 ** 60, 52), (3e20, 60)])
def test_append_scale_ends(value, e):
    cache = kvq.PagedCache.zeros(1, 1, 1, 16, 64)
    k = torch.full((1, 1, 64), value, dtype=torch.bfloat16, device="cuda")
    kvq.pages_append(cache, k, -k, dev([[0]]), dev([1]))
    clean()
    want = P.scale_exponent(abs(float(k[0, 0, 0])))
    assert want == e and exps_of(cache.k_scale)[0, 0, 0] == e
    got = cache.k_codes.float()[0, 0, 0, 0, 0].item()
    assert got == P.e4m3_round(float(k[0, 0, 0]) * 2.0 ** -e)
    assert cache.v_codes.float()[0, 0, 0, 0, 0].item() == -got


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 1e38])
def test_append_out_of_range_is_recorded(bad):
    cache = kvq.PagedCache.zeros(1, 2, 1, 16, 64)
    k = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    v[0, 0, 5] = bad
    kvq.pages_append(cache, k, v, dev([[1]]), dev([1]))
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_ERR_RANGE
    assert kvq.last_device_status() == kvq.KVQ_OK


# ---- attention ----

ATTENTION = [  # d, page, q heads, cache heads, lengths, query rows, causal, window
    (128, 16, 1, 1, [1], [1], True, 0),
    (64, 16, 3, 3, [5, 16, 17], [1, 1, 1], True, 0),
    (128, 64, 8, 2, [300, 1, 64, 0, 65], [1, 1, 1, 1, 1], True, 0),
    (128, 32, 10, 2, [513, 100], [1, 1], False, 0),
    (64, 128, 16, 1, [1000, 3], [1, 1], True, 100),
    (128, 16, 14, 2, [700, 30, 250], [1, 1, 1], True, 33),
    (128, 64, 32, 1, [200], [1], True, 0),
    (64, 32, 8, 4, [90, 40, 33], [4, 2, 7], True, 0),
    (128, 64, 6, 2, [500, 3, 130], [5, 5, 0], True, 64),        # rows before the first key
    (128, 16, 4, 4, [130], [3], False, 0),
    (128, 64, 4, 2, [300, 129], [300, 70], True, 0),
    (64, 64, 4, 4, [260], [129], False, 0),
    (128, 32, 5, 1, [400, 77, 20], [90, 77, 33], True, 50),
    (128, 128, 2, 2, [257, 1], [128, 1], False, 0),
    (64, 16, 7, 1, [333], [61], True, 17),
    (128, 16, 2, 1, [40], [150], True, 0),                      # more rows than keys
    (64, 128, 24, 8, [150, 300], [1, 65], False, 90),
    (128, 64, 3, 1, [640], [1], True, 1),
    (64, 32, 8, 1, [3000, 2000], [5, 5], True, 0),              # one row tile, many key tiles
    (128, 64, 2, 1, [2500], [50], False, 2100),
    (128, 128, 2, 1, [1900], [140], True, 0),
]


def pool_case(seed, lens, page, heads, d, **kw):
    rng = np.random.default_rng(seed)
    n_pages = sum(-(-n // page) for n in lens) + 2
    codes, exps = random_pool(seed, 1, n_pages, heads, page, d, **kw)
    table = make_table(rng, lens, page, n_pages)
    return rng, codes, exps, table


@pytest.mark.parametrize("d,page,hq,hkv,lens,counts,causal,window", ATTENTION)
def test_attention(d, page, hq, hkv, lens, counts, causal, window):
    rng, codes, exps, table = pool_case(d + sum(lens), lens, page, hkv, d, e_lo=-9, e_hi=-5)
    q = rows_of(rng, sum(counts), hq, d, 0.3)
    # whatever the last pages hold behind the lengths must not matter
    codes = [c.clone() for c in codes]
    for b, n in enumerate(lens):
        if n % page:
            for c in codes:
                c[0, table[b][n // page], :, n % page:] = 0x7F
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ref = P.attention(pool, q.double().numpy(), table, lens, counts, 1 / np.sqrt(d), causal, window)
    cache = cache_of(codes, exps)
    one = all(n == 1 for n in counts)
    for off in ([offsets_of(counts)] + ([None] if one else [])):
        got = kvq.paged_attention(cache, q.cuda(), dev(table), dev(lens), off, causal=causal, window=window,
                                  with_lse=True, max_q=max(counts))
        clean()
        check_attention(got, ref, d, max(lens), str((lens, counts)))


@pytest.mark.parametrize("d,hq,hkv,rows", [(128, 4, 2, 1), (64, 6, 1, 3), (128, 2, 2, 40)])
def test_attention_strides_layer_and_stale_pages(d, hq, hkv, rows):
    """Heads before rows, a layer other than the first, a table cut out of a
    wider one, NaN in every page and entry that is not the sequences'."""
    lens, page = [100, 37], 16
    rng, codes, exps, table = pool_case(5, lens, page, hkv, d, e_lo=-8, e_hi=-6)
    mine = {int(x) for r in table for x in r if x >= 0}
    full = [torch.full((3,) + tuple(c.shape[1:]), 0x7F, dtype=torch.uint8) for c in codes]
    for f, c in zip(full, codes):
        for i in mine:
            f[1, i] = c[0, i]
    ex = [np.repeat(e, 3, 0) for e in exps]
    cache = cache_of(full, ex)
    q = rows_of(rng, 2 * rows, hq, d, 0.2)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ref = P.attention(pool, q.double().numpy(), table, lens, [rows] * 2, 0.2, True, 0)
    qs = q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    wide = torch.full((2, table.shape[1] + 5), 1 << 30, dtype=torch.int32)
    wide[:, :table.shape[1]] = torch.from_numpy(table)
    wide[torch.from_numpy(np.pad(table, ((0, 0), (0, 5)), constant_values=-1) < 0)] = 1 << 30
    got = kvq.paged_attention(cache, qs, wide.cuda()[:, 0:table.shape[1] + 2], dev(lens), offsets_of([rows] * 2),
                              scale=0.2, layer=1, with_lse=True, max_q=rows)
    clean()
    check_attention(got, ref, d, 100)


@pytest.mark.parametrize("d,page,hq,rows", [(128, 16, 4, 1), (64, 16, 2, 5), (64, 64, 4, 1), (128, 32, 8, 20),
                                            (64, 16, 6, 30), (128, 128, 2, 300)])
def test_attention_pages_before_the_window_may_be_gone(d, page, hq, rows):
    """Table entries of pages wholly before every row's window are not read."""
    lens, window = [520, 600, 40], 45
    rng, codes, exps, table = pool_case(31, lens, page, 2, d, e_lo=-8, e_hi=-6)
    counts = [rows, rows, min(rows, 3)]
    q = rows_of(rng, sum(counts), hq, d, 0.2)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ref = P.attention(pool, q.double().numpy(), table, lens, counts, 0.1, True, window)
    t = table.copy()
    for b, (n, r) in enumerate(zip(lens, counts)):
        t[b, :max(0, n - r - window + 1) // page] = -1 if b else 1 << 30
    got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(t), dev(lens), offsets_of(counts), scale=0.1,
                              window=window, with_lse=True, max_q=max(counts))
    clean()
    check_attention(got, ref, d, window)


@pytest.mark.parametrize("rows,hq", [(1, 2), (2, 2), (80, 2)])
def test_attention_wide_scales(rows, hq):
    """Value pages 40 binades apart: the large page decides the output, the
    small one still counts in the softmax; and the other way round."""
    d, page, lens = 64, 16, [64]
    for order in (1, -1):
        rng, codes, exps, table = pool_case(9, lens, page, 1, d, e_lo=-8, e_hi=-8)
        for i, p in enumerate(table[0]):
            exps[1][0, p, :] = [-50, -10, -30, 0][::order][i]
        q = rows_of(rng, rows, hq, d, 0.2)
        pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
        ref = P.attention(pool, q.double().numpy(), table, lens, [rows], 0.02, False, 0)
        cache = cache_of(codes, exps)
        got = kvq.paged_attention(cache, q.cuda(), dev(table), dev(lens), offsets_of([rows]), scale=0.02, causal=False,
                                  with_lse=True, max_q=rows)
        clean()
        check_attention(got, ref, d, 64)


@pytest.mark.parametrize("rows", [1, 3, 64])
def test_attention_large_scores(rows):
    """Scores of some hundreds: one key takes everything."""
    d, lens, page = 128, [200], 32
    rng, codes, exps, table = pool_case(11, lens, page, 1, d, e_lo=-4, e_hi=-4)
    q = rows_of(rng, rows, 4, d, 0.1)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ref = P.attention(pool, q.double().numpy(), table, lens, [rows], 1.0, True, 0)
    got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), offsets_of([rows]), scale=1.0,
                              with_lse=True, max_q=rows)
    clean()
    check_attention(got, ref, d, 200)


@pytest.mark.parametrize("counts", [[1, 1], [6, 40]])
def test_attention_bad_pages_are_skipped_and_recorded(counts):
    """A table entry outside the pool: recorded, its tokens left out, the
    other sequence untouched by it."""
    d, page, lens = 128, 16, [100, 100]
    rng, codes, exps, table = pool_case(13, lens, page, 2, d, e_lo=-8, e_hi=-6)
    n_pages = codes[0].shape[1]
    q = rows_of(rng, sum(counts), 2, d, 0.2)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ref = P.attention(pool, q.double().numpy(), table, lens, counts, 0.1, True, 0)
    for wrong in (-1, n_pages, 1 << 30):
        t = table.copy()
        t[0, 3] = wrong
        got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(t), dev(lens), offsets_of(counts), scale=0.1,
                                  with_lse=True, max_q=max(counts))
        torch.cuda.synchronize()
        assert kvq.last_device_status() == kvq.KVQ_ERR_PAGE
        r = counts[0]
        check_attention([g[r:] for g in got], [x[r:] for x in ref], d, 100)
        assert torch.isfinite(got[0]).all()


def test_lengths_and_offsets_outside_are_recorded():
    d, page = 64, 16
    codes, exps = random_pool(1, 1, 4, 1, page, d)
    cache = cache_of(codes, exps)
    q = torch.ones(2, 1, d, dtype=torch.bfloat16, device="cuda")
    table = dev([[0, 1], [2, 3]])
    for lens, off, max_q in (([40, 16], None, None), ([-1, 16], None, None), ([16, 16], [0, 3, 2], None),
                             ([16, 16], [-1, 1, 2], None), ([16, 16], [0, 2, 2], 1)):
        kvq.paged_attention(cache, q, table, dev(lens), None if off is None else dev(off), max_q=max_q)
        torch.cuda.synchronize()
        assert kvq.last_device_status() == kvq.KVQ_ERR_PAGE, (lens, off)
    before = codes_of(cache.k_codes).copy()
    for lens, off in (([40, 0], [0, 2, 2]), ([1, 16], [0, 2, 2])):      # beyond the table; more rows than the length
        kvq.pages_append(cache, q, q, table, dev(lens), dev(off))
        torch.cuda.synchronize()
        assert kvq.last_device_status() == kvq.KVQ_ERR_PAGE, (lens, off)
    kvq.pages_append(cache, q, q, dev([[9, 9], [-3, 9]]), dev([5, 5]))
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_ERR_PAGE
    assert np.array_equal(codes_of(cache.k_codes)[0, 2:], before[0, 2:])


def test_nothing_to_do():
    cache = kvq.PagedCache.zeros(1, 4, 2, 16, 64)
    empty = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    table, lens = dev(np.zeros((0, 3))), dev(np.zeros(0))
    kvq.pages_append(cache, empty, empty, table, lens)
    assert kvq.paged_attention(cache, empty, table, lens).shape == (0, 2, 64)
    kvq.pages_copy(cache, [], [])
    t, n = kvq.pages_compact(cache, table)
    assert t.shape == (0, 3) and int(n) == 0
    # sequences without a token, and without a row
    q = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = kvq.paged_attention(cache, q, dev([[0], [1]]), dev([0, 0]), with_lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()
    out, lse = kvq.paged_attention(cache, q, dev(np.zeros((2, 0))), dev([0, 0]), with_lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()
    clean()


# ---- copy, compact ----

@pytest.mark.parametrize("layers,n_pages,heads,page,d,n", [(1, 4, 1, 16, 64, 1), (3, 50, 2, 16, 64, 20),
                                                            (2, 1400, 1, 16, 64, 700), (5, 9, 5, 128, 128, 3)])
def test_copy(layers, n_pages, heads, page, d, n):
    rng = np.random.default_rng(n)
    codes, exps = random_pool(2, layers, n_pages, heads, page, d)
    cache = cache_of(codes, exps)
    ids = rng.permutation(n_pages)
    dst, src = ids[:n], rng.choice(ids[n:], n)          # a page may be copied to several
    kvq.pages_copy(cache, src.tolist(), torch.from_numpy(dst))
    clean()
    for kv, (c, s) in enumerate(((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale))):
        want, e = codes[kv].numpy().copy(), exps[kv].copy()
        want[:, dst], e[:, dst] = want[:, src], e[:, src]
        assert np.array_equal(codes_of(c), want) and np.array_equal(exps_of(s), e)


@pytest.mark.parametrize("layers,n_pages,batch,width,share", [
    (1, 1, 1, 1, 1.0), (2, 40, 3, 7, 0.5), (1, 33, 2, 20, 0.9), (1, 64, 1, 64, 1.0), (3, 70, 4, 5, 0.0),
    (1, 5000, 7, 400, 0.4), (1, 40000, 30, 700, 0.45)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(layers, n_pages, batch, width, share, in_place):
    rng = np.random.default_rng(n_pages + batch)
    codes, exps = random_pool(4, layers, min(n_pages, 64), 1, 16, 64)
    codes = [c.repeat(1, -(-n_pages // 64) if n_pages > 64 else 1, 1, 1, 1)[:, :n_pages].contiguous() for c in codes]
    exps = [rng.integers(-9, 9, (layers, n_pages, 1)) for _ in range(2)]
    table = np.where(rng.random((batch, width)) < share, rng.integers(0, n_pages, (batch, width)), -1).astype(np.int32)
    want, n_live, moves = P.compact(table, n_pages)
    cache = cache_of(codes, exps)
    wide = torch.full((batch, width + 4), 3, dtype=torch.int32, device="cuda")
    wide[:, :width] = dev(table)
    t, n = kvq.pages_compact(cache, wide[:, :width], out=wide[:, :width] if in_place else None)
    clean()
    assert int(n) == n_live and np.array_equal(t.cpu().numpy(), want)
    assert (wide[:, width:] == 3).all()
    for kv, (c, s) in enumerate(((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale))):
        w, e = codes[kv].numpy().copy(), exps[kv].copy()
        for a, b in moves:
            w[:, b], e[:, b] = w[:, a], e[:, a]
        assert np.array_equal(codes_of(c), w) and np.array_equal(exps_of(s), e)


def test_compact_entries_outside_are_recorded():
    cache = kvq.PagedCache.zeros(1, 8, 1, 16, 64)
    t, n = kvq.pages_compact(cache, dev([[7, 8, 1 << 30, -5]]))
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_ERR_PAGE
    assert t.tolist() == [[0, 8, 1 << 30, -5]] and int(n) == 1


# ---- together ----

def test_serving_run():
    """Two prompts in, decode, one forks (its full pages shared, its tail page
    copied), all decode, one ends and the pool is compacted; every step's
    attention against the oracle, which runs the same steps."""
    rng = np.random.default_rng(7)
    layers, n_pages, heads, hq, page, d = 2, 40, 2, 6, 16, 64
    cache = kvq.PagedCache.zeros(layers, n_pages, heads, page, d)
    pools = [P.Pool([np.zeros((n_pages, heads, page, d), np.uint8)] * 2, [np.zeros((n_pages, heads))] * 2)
             for _ in range(layers)]
    free = list(rng.permutation(n_pages))
    tables, lens = [[], []], [0, 0]

    def step(counts, causal=True):
        for b, n in enumerate(counts):
            lens[b] += n
            while len(tables[b]) * page < lens[b]:
                tables[b].append(int(free.pop()))
        t = np.full((len(lens), max(map(len, tables))), -1, np.int32)
        for b, r in enumerate(tables):
            t[b, :len(r)] = r
        one = all(n == 1 for n in counts)
        off = None if one else offsets_of(counts)
        for layer in range(layers):
            k, v = rows_of(rng, sum(counts), heads, d, 0.5), rows_of(rng, sum(counts), heads, d, 0.5)
            q = rows_of(rng, sum(counts), hq, d, 0.2)
            kvq.pages_append(cache, k.cuda(), v.cuda(), dev(t), dev(lens), off, layer=layer)
            got = kvq.paged_attention(cache, q.cuda(), dev(t), dev(lens), off, layer=layer, with_lse=True,
                                      max_q=max(counts))
            P.append(pools[layer], k.double().numpy(), v.double().numpy(), t, lens, counts)
            ref = P.attention(pools[layer], q.double().numpy(), t, lens, counts, 1 / np.sqrt(d), True, 0)
            clean()
            check_attention(got, ref, d, max(lens))
        return t

    step([70, 23])
    for _ in range(3):
        step([1, 1])
    # fork sequence 0
    tail = tables[0][-1]
    new = int(free.pop())
    kvq.pages_copy(cache, [tail], [new])
    for p in pools:
        for kv in range(2):
            p.val[kv][new], p.exp[kv][new] = p.val[kv][tail], p.exp[kv][tail]
    tables.append(tables[0][:-1] + [new])
    lens.append(lens[0])
    for _ in range(3):
        step([1, 1, 1])
    step([4, 0, 9])
    # sequence 1 ends
    del tables[1], lens[1]
    t = step([1, 1])
    out, n_live = kvq.pages_compact(cache, dev(t))
    want, n, moves = P.compact(t, n_pages)
    assert int(n_live) == n and np.array_equal(out.cpu().numpy(), want)
    for p in pools:
        for kv in range(2):
            for a, b in moves:
                p.val[kv][b], p.exp[kv][b] = p.val[kv][a], p.exp[kv][a]
    tables = [[int(x) for x in r if x >= 0] for r in out.cpu().numpy()]
    free = list(range(n, n_pages))
    for _ in range(2):
        step([1, 1])


def test_step_in_a_graph_follows_lengths_and_tables():
    """One decode step captured, replayed as lengths, tables and rows change."""
    rng = np.random.default_rng(3)
    n_pages, heads, hq, page, d = 20, 2, 4, 16, 128
    codes, exps = random_pool(8, 1, n_pages, heads, page, d, e_lo=-8, e_hi=-6)
    cache = cache_of(codes, exps)
    table, lens = torch.zeros(2, 9, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    k, v, q = (torch.zeros(2, h, d, dtype=torch.bfloat16, device="cuda") for h in (heads, heads, hq))
    table.copy_(dev([[0] * 9, [1] * 9]))
    ws = torch.empty(cache.workspace_bytes(hq, 2, 9, 2, 1), dtype=torch.uint8, device="cuda")

    def run():
        kvq.pages_append(cache, k, v, table, lens)
        return kvq.paged_attention(cache, q, table, lens, with_lse=True, workspace=ws)
    run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for lengths in ([140, 3], [16, 17], [1, 100]):
        t = make_table(rng, lengths, page, n_pages, width=9)
        cache.k_codes.view(torch.uint8).copy_(codes[0])
        cache.v_codes.view(torch.uint8).copy_(codes[1])
        for dst, e in ((cache.k_scale, exps[0]), (cache.v_scale, exps[1])):
            dst.copy_(torch.from_numpy(2.0 ** np.asarray(e, np.float64)).to(torch.bfloat16))
        table.copy_(dev(t))
        lens.copy_(dev(lengths))
        kk, vv, qq = rows_of(rng, 2, heads, d, 0.4), rows_of(rng, 2, heads, d, 0.4), rows_of(rng, 2, hq, d, 0.2)
        k.copy_(kk), v.copy_(vv), q.copy_(qq)
        g.replay()
        clean()
        pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
        P.append(pool, kk.double().numpy(), vv.double().numpy(), t, lengths, [1, 1])
        check_attention(got, P.attention(pool, qq.double().numpy(), t, lengths, [1, 1], 1 / np.sqrt(d), True, 0), d, 140)


def test_two_streams_at_once():
    """Calls on two streams, each with its own outputs and workspace."""
    rng, codes, exps, table = pool_case(21, [900, 800], 64, 2, 128, e_lo=-8, e_hi=-6)
    cache = cache_of(codes, exps)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    qs = [rows_of(rng, 2, 8, 128, 0.2) for _ in range(2)]
    t, lens = dev(table), dev([900, 800])
    dq = [q.cuda() for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(kvq.paged_attention(cache, dq[i], t, lens, with_lse=True, stream=streams[i]))
    clean()
    for i in range(2):
        ref = P.attention(pool, qs[i].double().numpy(), table, [900, 800], [1, 1], 1 / np.sqrt(128), True, 0)
        for g in got[i]:
            check_attention(g, ref, 128, 900)
            assert torch.equal(g[0], got[i][0][0]) and torch.equal(g[1], got[i][0][1])
