"""Attention with shaped scores over batches that are mostly padding: whole row
tiles, thousands of rows, that attend to nothing beside rows that do."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from quantized_kv_cache_quantize_gb300 import kvq
from tests.paged_common import cache_of, dev, offsets_of
from tests.test_gpu_scored import check, clean, pool_case, rows_of

pytestmark = pytest.mark.gpu

PADDED = [  # d, page, q heads, cache heads, live rows, all rows
    (128, 128, 32, 8, 40, 3500),
    (64, 64, 32, 8, 70, 4133),
    (128, 64, 8, 8, 5, 3000),
    (64, 128, 24, 2, 300, 2500),
]


@pytest.mark.parametrize("d,page,hq,hkv,live,rows", PADDED)
@pytest.mark.parametrize("softcap,slope", [(5.0, 0.0), (0.0, 0.01), (5.0, 0.01), (0.0, 0.0)])
def test_tiles_of_rows_that_see_nothing(d, page, hq, hkv, live, rows, softcap, slope):
    """A padding row is zero and -infinity whatever its query holds, however its
    CTA's query loads come back: queries of every size, cold in the caches, the
    output full of other numbers before, many times over; the live rows are the
    oracle's and the same bits every time."""
    length = rows + 100
    rng, codes, exps, table = pool_case(d + rows, [length], page, hkv, d, e_lo=-9, e_hi=-6)
    q = rows_of(rng, rows, hq, d, spread=1.0, heat=4.0)
    ranges = np.tile([[7, 7]], (rows, 1))
    ranges[:live] = np.stack([rng.integers(0, 40, live), rng.integers(41, length, live)], 1)
    s = np.full(hq, slope, np.float32)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ref = P.attention_scored(pool, q[:live].double().numpy(), table, [length], [live], 0.1, False, 0, softcap,
                             ranges=ranges[:live])
    if slope:   # (positions count from the whole batch's first row)
        t0 = length - rows
        full = P.attention_scored(pool, q[:live].double().numpy(), table, [t0 + live], [live], 0.1, False, 0, softcap, s,
                                  ranges=np.minimum(ranges[:live], t0 + live))
        ranges[:live] = np.minimum(ranges[:live], t0 + live)
        ref = full
    # the rows apart from one another in memory, as slices of a wider projection
    wide = torch.empty(rows, hq + 8, d, dtype=torch.bfloat16, device="cuda")
    wide[:, :hq] = q.cuda()
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")   # more than L2 holds
    cache, t, n, off, r = cache_of(codes, exps), dev(table), dev([length]), offsets_of([rows]), dev(ranges)
    out = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")
    first = None
    for turn in range(12):
        out.fill_(7.0)
        if turn % 2 == 0:
            cold.fill_(turn)
        _, lse = kvq.paged_attention(cache, wide[:, :hq], t, n, off, scale=0.1, causal=False, with_lse=True, max_q=rows,
                                     softcap=softcap, slopes=dev(s, torch.float32), ranges=r, out=out)
        clean()
        assert (out[live:] == 0).all() and (lse[live:] == -np.inf).all(), turn
        if first is None:
            first = out[:live].clone(), lse[:live].clone()
            check(first, ref, d, length, softcap)
        assert torch.equal(out[:live], first[0]) and torch.equal(lse[:live], first[1]), turn


def test_nobody_sees_anything():
    """A batch whose every range is empty, in sequences of several lengths, one of
    them without a token."""
    rng, codes, exps, table = pool_case(3, [900, 1, 2000, 0], 64, 4, 128, e_lo=-9, e_hi=-6)
    counts = [900, 1, 1500, 0]
    rows = sum(counts)
    q = rows_of(rng, rows, 16, 128, spread=1.0, heat=4.0).cuda()
    for softcap in (0.0, 3.0):
        for _ in range(6):
            out = torch.full_like(q, 7.0)
            _, lse = kvq.paged_attention(cache_of(codes, exps), q, dev(table), dev([900, 1, 2000, 0]), offsets_of(counts),
                                         with_lse=True, max_q=1500, softcap=softcap, out=out,
                                         ranges=torch.zeros(rows, 2, dtype=torch.int32, device="cuda"))
            clean()
            assert (out == 0).all() and (lse == -np.inf).all()
