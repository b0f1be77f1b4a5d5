"""Rotations among views of one allocation: outputs between other tensors' heads,
rows and batch entries are written, outputs over them refused."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from quantized_kv_cache_quantize_gb300 import kvq
from tests.paged_common import dev
from tests.test_gpu_rope import bits, clean, rows_of, table_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 9, 700])
def test_outputs_between_other_heads(rows):
    rng = np.random.default_rng(rows)
    t = table_of(1000, 64, None, False)
    pos = dev(rng.integers(0, 1000, rows))
    wide = rows_of(rng, rows, 80, 128).cuda()
    q, k, q_out, k_out = wide[:, :32], wide[:, 40:48], wide[:, 48:80], wide[:, 32:40]
    want = kvq.rope(t, q.clone(), pos, k=k.clone())
    before = wide.clone()
    kvq.rope(t, q, pos, k=k, q_out=q_out, k_out=k_out)
    clean()
    assert np.array_equal(bits(q_out), bits(want[0])) and np.array_equal(bits(k_out), bits(want[1]))
    assert torch.equal(q, before[:, :32]) and torch.equal(k, before[:, 40:48])
    for qo, ko in ((wide[:, 8:40], k_out), (wide[:, 1:33], None), (q_out, wide[:, 31:39]), (q_out, wide[:, 47:55]), (q_out, wide[:, 48:56])):
        with pytest.raises(kvq.KVQError) as e:
            kvq.rope(t, q, pos, k=k, q_out=qo, k_out=ko)
        assert e.value.status == kvq.KVQ_ERR_INVALID_ARG
    assert torch.equal(q, before[:, :32])


def test_outputs_between_other_heads_of_the_window():
    rng = np.random.default_rng(5)
    batch, rows = 2, 50
    t = table_of(64, 32, [16, 8, 8], True)
    pos = dev(rng.integers(0, 64, (rows, 3)))
    x = rows_of(rng, batch, 12, rows, 64).cuda()
    want = kvq.rope(t, x[:, :4].contiguous(), pos, k=x[:, 4:6].contiguous())
    kvq.rope(t, x[:, :4], pos, k=x[:, 4:6], q_out=x[:, 6:10], k_out=x[:, 10:])
    clean()
    assert np.array_equal(bits(x[:, 6:10]), bits(want[0])) and np.array_equal(bits(x[:, 10:]), bits(want[1]))
    with pytest.raises(kvq.KVQError):
        kvq.rope(t, x[:, :4], pos, k=x[:, 4:6], q_out=x[:, 5:9], k_out=x[:, 10:])


@pytest.mark.parametrize("offsets", [False, True])
def test_append_writes_queries_beside_its_inputs(offsets):
    rng = np.random.default_rng(8)
    rows, d = 6, 128
    t = table_of(100, 64, None, False)
    table = dev(np.arange(rows)[:, None]) if not offsets else dev([[0]])
    lens = dev([1] * rows) if not offsets else dev([rows])
    off = dev([0, rows]) if offsets else None
    wide = rows_of(rng, rows, 14, d).cuda()
    k, v, q, room = wide[:, :2], wide[:, 2:4], wide[:, 4:8], wide[:, 8:12]
    cache = kvq.PagedCache.zeros(1, 8, 2, 16, d)
    want = kvq.pages_append_rope(cache, t, k, v, table, lens, off, q=q).clone()
    got = kvq.pages_append_rope(cache, t, k, v, table, lens, off, q=q, q_out=room)
    clean()
    assert np.array_equal(bits(got), bits(want))
    for bad in (wide[:, 1:5], wide[:, 3:7], wide[:, 5:9], wide[:, :4]):
        with pytest.raises(kvq.KVQError) as e:
            kvq.pages_append_rope(cache, t, k, v, table, lens, off, q=q, q_out=bad)
        assert e.value.status == kvq.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("offsets,lens", [(None, [0, 3]), ([0, 5], [2]), ([0, 40, 41], [7, 1])])
def test_more_rows_than_tokens_is_one_error(offsets, lens):
    """Rows before their sequence's first token have no place: the length is what is
    wrong, whichever of the keys' and the queries' blocks comes first."""
    rng = np.random.default_rng(9)
    rows = offsets[-1] if offsets else len(lens)
    t = table_of(100, 64, None, False)
    table = dev(np.arange(2 * len(lens)).reshape(len(lens), 2))
    x = rows_of(rng, rows, 12, 128).cuda()
    for _ in range(30):
        cache = kvq.PagedCache.zeros(1, 8, 2, 16, 128)
        y = kvq.pages_append_rope(cache, t, x[:, :2], x[:, 2:4], table, dev(lens), dev(offsets) if offsets else None, q=x[:, 4:])
        torch.cuda.synchronize()
        assert kvq.last_device_status() == kvq.KVQ_ERR_PAGE
        first = 0 if offsets is None else offsets[1] - lens[0]     # the row of token 0, or of none
        assert np.array_equal(bits(y[:first + 1]), bits(x[:first + 1, 4:]))     # as they are, at place 0
