"""Capped scores whose raw products of codes are as large as they get: rows and
keys of one magnitude and the same signs, so that the factor from a raw score to
the cap is tiny where the score still lies well inside the cap."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from quantized_kv_cache_quantize_gb300 import kvq
from tests.paged_common import cache_of, dev, offsets_of
from tests.test_gpu_scored import check, clean, pool_case, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,rows", [(2, 1), (1, 40), (1, 300)])
@pytest.mark.parametrize("softcap", [2.0 ** -12, 5.0, 15.0, 30.0, 50.0, 500.0])
@pytest.mark.parametrize("x", [0.3, 0.36, 0.399, 0.7])
@pytest.mark.parametrize("masked", [False, True])
def test_scores_of_flat_rows(d, hq, rows, softcap, x, masked):
    """Raw scores of 5e6 to 1.3e7 at x of the cap: the query 1.75 with signs (224 as
    a code, exact), the keys' codes 384, 416 and 448 with the same signs.  The
    tolerance is that of every capped score (check): 2^-20 of the cap beside the
    rounding of the sum of products; a coefficient lost to fp32's range is off by
    2^-14 of it."""
    n, page = (300 if masked else 256), 64
    rng, codes, exps, table = pool_case(5, [n], page, 1, d, e_lo=-8, e_hi=-8)
    sign = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    k = rng.choice([384.0, 416.0, 448.0], (exps[0].shape[1], 1, page, 1)) * sign
    codes[0][0] = torch.from_numpy(P.e4m3_code(k))
    q = torch.from_numpy(np.broadcast_to(1.75 * sign, (rows, hq, d)).copy()).bfloat16()
    scale = float(np.float32(x * softcap / (1.75 * 1.75 * d)))
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    ref = P.attention_scored(pool, q.double().numpy(), table, [n], [rows], scale, masked, 0, softcap)
    got = kvq.paged_attention(cache_of(codes, exps), q.cuda(), dev(table), dev([n]), offsets_of([rows]), scale=scale,
                              causal=masked, with_lse=True, max_q=rows, softcap=softcap)
    clean()
    # the codes' products are whole numbers below 2^24: summed without a rounding,
    # and the query has no part that is lost
    out, lse, bound, serr, qerr, herr, top = ref
    check(got, (out, lse, bound, serr * (8.0 / (d + 4)), 0 * qerr, herr, top), d, n, softcap)
