"""What masked places hold beside capped scores: no bit of any row's result."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from quantized_kv_cache_quantize_gb300 import kvq
from tests.paged_common import cache_of, dev, offsets_of
from tests.test_gpu_scored import check, clean, pool_case, rows_of

pytestmark = pytest.mark.gpu

HELD = {"zero": (0x00, 0), "large": (0x7E, 0), "minus": (0xFE, 0), "nan": (0x7F, 0), "scaled": (0x7E, 40), "small": (0x30, -40)}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,rows", [(2, 1), (2, 40), (2, 200)])
@pytest.mark.parametrize("softcap", [50.0, 600.0])
@pytest.mark.parametrize("slope", [0.0, 0.01])
def test_masked_places_decide_no_bit(d, hq, rows, softcap, slope):
    """Keys that no row attends to (behind the length, between ranges) hold zeros,
    the largest codes or NaN, a page between the ranges another scale; the results
    have the same bits.  Queries of one sign so that the largest codes' scores lie
    far beyond the cap."""
    page, n, lens = 64, 500, [437]
    rng, codes, exps, table = pool_case(31, [n], page, 1, d, e_lo=-8, e_hi=-6)
    q = rows_of(rng, rows, hq, d).abs()
    ranges = np.tile([[10, 150]], (rows, 1))
    ranges[1::2] = [[301, 437]]
    seen = np.zeros(n, bool)
    for lo, hi in ranges:
        seen[lo:hi] = True
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ref = P.attention_scored(pool, q.double().numpy(), table, lens, [rows], 0.1, False, 0, softcap, np.full(hq, slope), ranges=ranges)
    results = []
    for held, e in HELD.values():
        c2, e2 = [c.clone() for c in codes], [x.copy() for x in exps]
        for x in e2:
            x[0, table[0][3]] += e                                             # keys 192 to 255: nobody's
        for j in np.flatnonzero(~seen):
            for c in c2:
                c[0, table[0][j // page], :, j % page] = held
        got = kvq.paged_attention(cache_of(c2, e2), q.cuda(), dev(table), dev(lens), offsets_of([rows]), scale=0.1,
                                  causal=False, with_lse=True, max_q=rows, softcap=softcap, ranges=dev(ranges),
                                  slopes=dev(np.full(hq, slope), torch.float32) if slope else None)
        clean()
        results.append(got)
    check(results[0], ref, d, n, softcap)
    for held, got in zip(HELD, results):
        for a, b in zip(got, results[0]):
            assert torch.equal(a, b), (held, int((a != b).sum()), float((a.float() - b.float()).abs().max()))


@pytest.mark.parametrize("d,hq", [(64, 2), (128, 4)])
@pytest.mark.parametrize("heat", [1.0, 20.0])
@pytest.mark.parametrize("lo,hi", [(102, 131), (101, 130), (96, 128), (111, 112)])
@pytest.mark.parametrize("softcap,slope", [(6.0, 0.0), (0.0, 0.01), (6.0, 0.01)])
def test_one_row_beside_masked_neighbours(d, hq, heat, lo, hi, softcap, slope):
    """A single row, the decoding form: NaN in every key and value beside those of
    its range, which begins and ends at odd and even places."""
    page, lens = 32, [500]
    rng, codes, exps, table = pool_case(12, lens, page, 2, d, e_lo=-9, e_hi=-6)
    q = rows_of(rng, 1, hq, d, heat=heat)
    s = np.full(hq, slope, np.float32)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ref = P.attention_scored(pool, q.double().numpy(), table, lens, [1], 0.2, False, 0, softcap, s, ranges=np.array([[lo, hi]]))
    assert np.isfinite(ref[1]).all()
    codes = [c.clone() for c in codes]
    for j in list(range(lo)) + list(range(hi, 500)):
        for c in codes:
            c[0, table[0][j // page], :, j % page] = 0x7F
    for off in (offsets_of([1]), None):
        got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev(lens), off, scale=0.2, causal=False,
                                  with_lse=True, max_q=1, softcap=softcap, slopes=dev(s, torch.float32), ranges=dev([[lo, hi]]))
        clean()
        check(got, ref, d, hi - lo, softcap, str(off))
