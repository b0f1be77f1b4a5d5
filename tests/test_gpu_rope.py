"""Rotary positions on the GPU: the table against 64 bits, the rotation against
the 64-bit oracle and bit for bit against its fp32 steps, the append that
rotates against an append of rotated rows."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from quantized_kv_cache_quantize_gb300 import kvq
from tests.paged_common import cache_of, codes_of, dev, exps_of, make_table, offsets_of, random_pool

pytestmark = pytest.mark.gpu


def clean():
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_OK


def rows_of(rng, *shape, spread=0.5):
    x = rng.standard_normal(shape) * np.exp(rng.standard_normal(shape[:-1] + (1,)) * spread)
    return torch.from_numpy(x).float().bfloat16()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def table_of(n, pairs, sections, interleaved):
    return kvq.RopeTable.build(n, kvq.rope_frequencies(pairs, sections=sections if interleaved else None), sections, interleaved)


def axis_of(t):
    return list(t.struct.axis)[:t.pairs]


SHAPES = [  # d, pairs, sections, interleaved
    (128, 64, None, False),
    (128, 64, [22, 21, 21], True),
    (128, 32, [16, 8, 8], False),
    (128, 56, None, True),
    (64, 32, [8, 8, 8, 8], False),
    (64, 24, [23, 1], False),
    (64, 8, None, True),
]


# ---- the table ----

@pytest.mark.parametrize("n,pairs,factor", [(1, 8, 1.0), (70000, 32, 1.0), (513, 64, 0.75)])
def test_table(n, pairs, factor):
    f = kvq.rope_frequencies(pairs, 500.0)
    t = kvq.RopeTable.build(n, f, factor=factor)
    clean()
    angle = np.arange(n)[:, None] * np.array(f)
    want = np.stack([np.cos(angle), np.sin(angle)], -1) * factor
    # half a step of fp32, and what 64 bits leave of an angle up to 70000 (2^-53 of it, twice)
    assert np.abs(t.cos_sin.cpu().numpy() - want).max() <= 2.0 ** -24 * factor + 70000 * 2.0 ** -51


# ---- the rotation ----

def check_rope(got, x, want, steps, what=""):
    """want in 64 bits: two products, their sum, the table (2^-24 of |x0| + |x1|
    each, which twice the row's largest bounds), then BF16, half a step of 2^-7."""
    y = got.double().cpu().numpy()
    top = np.abs(x).max(-1, keepdims=True)
    assert (np.abs(y - want) <= 2.0 ** -8 * np.abs(want) + 9 * 2.0 ** -24 * top + 1e-38).all(), what
    assert np.array_equal(bits(got), bits(torch.from_numpy(steps).bfloat16())), what


@pytest.mark.parametrize("d,pairs,sections,interleaved", SHAPES)
@pytest.mark.parametrize("rows,heads,kv_heads", [(1, 1, 1), (7, 5, 2), (301, 8, 3), (40, 33, 1)])
def test_packed(d, pairs, sections, interleaved, rows, heads, kv_heads):
    rng = np.random.default_rng(rows + d + pairs)
    t = table_of(300, pairs, sections, interleaved)
    f = kvq.rope_frequencies(pairs, sections=sections if interleaved else None)
    pos = rng.integers(0, 300, (rows, t.axes)).astype(np.int32)
    q, k = rows_of(rng, rows, heads, d), rows_of(rng, rows, kv_heads, d)
    wide = torch.zeros(rows, heads + kv_heads + 1, d, dtype=torch.bfloat16)       # one fused projection
    wide[:, :heads], wide[:, heads:-1] = q, k
    wide = wide.cuda()
    cs = t.cos_sin.cpu().numpy()
    for inverse in (False, True):
        got = kvq.rope(t, wide[:, :heads], dev(pos), k=wide[:, heads:-1], inverse=inverse)
        clean()
        for y, x in zip(got, (q, k)):
            x = x.float().numpy()
            check_rope(y, x, P.rope(x, pos, f, axis_of(t), interleaved, inverse),
                       P.rope_steps(x, cs, pos, axis_of(t), interleaved, inverse))
    one = kvq.rope(t, q.cuda(), dev(pos) if t.axes > 1 else dev(pos[:, 0]), inverse=True)
    assert np.array_equal(bits(one), bits(got[0]))
    # in place, of the fused rows, the rest of which stays
    rest = wide[:, -1].clone()
    a, b = wide[:, :heads], wide[:, heads:-1]
    assert kvq.rope(t, a, dev(pos), k=b, q_out=a, k_out=b, inverse=True)[0] is a
    clean()
    assert np.array_equal(bits(a), bits(got[0])) and np.array_equal(bits(b), bits(got[1])) and torch.equal(wide[:, -1], rest)


@pytest.mark.parametrize("d,pairs,sections,interleaved", SHAPES[:5])
@pytest.mark.parametrize("shared", [True, False])
def test_window_layout(d, pairs, sections, interleaved, shared):
    """[batch, heads, rows, d], contiguous as the chunk window takes it, with
    positions of the whole batch or of each entry."""
    rng = np.random.default_rng(d + pairs)
    batch, heads, rows = 2, 3, 157
    t = table_of(64, pairs, sections, interleaved)
    pos = rng.integers(0, 64, (batch, rows, t.axes)).astype(np.int32)
    if shared:
        pos[1] = pos[0]
    q, k = rows_of(rng, batch, heads, rows, d), rows_of(rng, batch, heads + 1, rows, d)
    got = kvq.rope(t, q.cuda(), dev(pos[0] if shared else pos), k=k.cuda())
    clean()
    cs = t.cos_sin.cpu().numpy()
    for y, x in zip(got, (q, k)):
        assert y.is_contiguous() and y.shape == x.shape
        for b in range(batch):
            want = P.rope_steps(x[b].transpose(0, 1).float().numpy(), cs, pos[b], axis_of(t), interleaved)
            assert np.array_equal(bits(y[b].transpose(0, 1)), bits(torch.from_numpy(want).bfloat16()))


def test_strides_of_positions_and_outputs():
    """Positions [axes, rows] (as some models keep them) and an output whose
    heads come first; what lies between its rows stays."""
    rng = np.random.default_rng(0)
    t = table_of(90, 32, [16, 8, 8], False)
    pos = dev(rng.integers(0, 90, (3, 50)))
    x = rows_of(rng, 50, 4, 64).cuda()
    want = kvq.rope(t, x, pos.T.contiguous())
    room = torch.full((4, 50, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out = room[:, :, 0].transpose(0, 1)
    assert kvq.rope(t, x, pos.T, q_out=out) is out
    clean()
    assert torch.equal(out, want) and (room[:, :, 1] == 3.0).all()


def test_inverse_is_the_gradient_and_undoes():
    """The product of any g with the rotated x is that of the inverse rotation of
    g with x: differences of a linear map, exact on powers of two."""
    rng = np.random.default_rng(3)
    t = table_of(1000, 64, [22, 21, 21], True)
    pos = dev(rng.integers(0, 1000, (20, 3)))
    x, g = rows_of(rng, 20, 2, 128).cuda(), rows_of(rng, 20, 2, 128).cuda()
    y, h = kvq.rope(t, x, pos).double(), kvq.rope(t, g, pos, inverse=True).double()
    # a BF16 rounding of each element of y and of h, 2^-8 of it
    scale = (y.abs() * g.double().abs()).sum() + (h.abs() * x.double().abs()).sum()
    assert ((y * g.double()).sum() - (h * x.double()).sum()).abs() <= (2.0 ** -8 + 2.0 ** -20) * scale
    back = kvq.rope(t, kvq.rope(t, x, pos), pos, inverse=True)
    # two BF16 roundings: the first of both channels of a pair, turned with them
    top = x.double().abs().amax(-1, keepdim=True)
    assert ((back.double() - x.double()).abs() <= 3 * 2.0 ** -8 * top).all()


@pytest.mark.parametrize("bad", [-1, 64, 2 ** 31 - 1, -2 ** 31])
def test_position_outside_the_table_is_recorded(bad):
    t = table_of(64, 32, [16, 16], False)
    x = rows_of(np.random.default_rng(0), 5, 2, 64).cuda()
    pos = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    pos[3, 1] = bad
    y = kvq.rope(t, x, pos)
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_ERR_POSITION
    assert kvq.last_device_status() == kvq.KVQ_OK
    pos[3, 1] = 0 if bad < 0 else 63
    assert torch.equal(y, kvq.rope(t, x, pos))


def test_not_finite_rows_stay_theirs():
    t = table_of(64, 32, None, False)
    x = rows_of(np.random.default_rng(0), 6, 2, 64)
    x[2, 1, 5], x[4, 0, 40] = float("inf"), float("nan")
    pos = dev(np.arange(6))
    y = kvq.rope(t, x.cuda(), pos).cpu()
    clean()
    want = torch.from_numpy(P.rope_steps(x.float().numpy(), t.cos_sin.cpu().numpy(), np.arange(6)[:, None], [0] * 32, False)).bfloat16()
    assert torch.equal(y.nan_to_num(7.0), want.nan_to_num(7.0)) and torch.isnan(y).sum() == torch.isnan(want).sum() > 0


def test_nothing_to_rotate():
    t = table_of(64, 32, None, False)
    for shape in ((0, 4, 64), (5, 0, 64), (2, 0, 3, 64), (0, 2, 3, 64)):
        x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        pos = torch.zeros(shape[0] if len(shape) == 3 else shape[2], 1, dtype=torch.int32, device="cuda")
        assert kvq.rope(t, x, pos).shape == shape
    clean()


def test_refusals_on_the_device():
    t = table_of(64, 32, [16, 16], False)
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    for bad in (pos[:, 0], pos[:4], pos.long(), pos.cpu(), pos[None]):
        with pytest.raises(ValueError, match="positions"):
            kvq.rope(t, x, bad)
    for bad in (x[:4], x.float(), x[..., :32], x[None]):
        with pytest.raises(ValueError):
            kvq.rope(t, x, pos, k=bad)
        with pytest.raises(ValueError):
            kvq.rope(t, x, pos, q_out=bad)
    with pytest.raises(ValueError, match="repeat"):
        kvq.rope(t, x, pos, q_out=x[:1].expand(5, 2, 64))
    y = x.clone()
    shared = [dict(q_out=x.as_strided((5, 2, 64), (64, 320, 1))), dict(k=y, q_out=x, k_out=x), dict(k=y, q_out=y),
              dict(k=y, k_out=x)]
    for kw in shared:                                             # in place, but other places; the other tensor's memory
        with pytest.raises(kvq.KVQError) as e:
            kvq.rope(t, x, pos, **kw)
        assert e.value.status == kvq.KVQ_ERR_INVALID_ARG
    assert torch.equal(kvq.rope(t, y[:1], pos[:1], q_out=y.as_strided((1, 2, 64), (4096, 64, 1))), kvq.rope(t, x[:1], pos[:1]))
    with pytest.raises(ValueError, match="contiguous channels"):
        kvq.rope(t, x.transpose(1, 2), pos)
    with pytest.raises(ValueError, match="without k"):
        kvq.rope(t, x, pos, k_out=x)
    with pytest.raises(kvq.KVQError) as e:
        kvq.rope(t, torch.zeros(5, 2, 68, dtype=torch.bfloat16, device="cuda")[..., :64], pos)   # rows of 136 bytes
    assert e.value.status == kvq.KVQ_ERR_ALIGNMENT
    clean()


# ---- the append ----

APPENDS = [  # d, page, heads, q_heads, pairs, sections, interleaved, lengths after, new rows
    (128, 16, 2, 2, 64, None, False, [1], [1]),
    (64, 16, 1, 4, 32, None, True, [16, 17, 31], [1, 1, 1]),
    (128, 64, 3, 6, 64, [22, 21, 21], True, [200, 1, 64, 65, 0], [200, 1, 64, 1, 0]),
    (64, 128, 2, 0, 16, None, False, [129, 300, 5], [2, 171, 0]),
    (128, 32, 5, 5, 32, [16, 8, 8], False, [100, 33, 32, 7, 64], [68, 33, 1, 7, 31]),
    (64, 32, 4, 8, 24, None, False, [40] * 9, [1] * 9),
    (128, 128, 1, 7, 56, [50, 6], True, [1000], [873]),
    (64, 16, 8, 8, 32, [8, 8, 8, 8], False, [63, 130], [1, 67]),
]


@pytest.mark.parametrize("d,page,heads,q_heads,pairs,sections,interleaved,lens,counts", APPENDS)
@pytest.mark.parametrize("strided", [False, True])
def test_append(d, page, heads, q_heads, pairs, sections, interleaved, lens, counts, strided):
    """Codes, scales and queries bit for bit: those of an append of the rows
    rotated in fp32."""
    rng = np.random.default_rng(sum(lens) + d + page)
    n_pages = sum(-(-n // page) for n in lens) + 2
    codes, exps = random_pool(3, 1, n_pages, heads, page, d, e_lo=-12, e_hi=-5)
    table = make_table(rng, lens, page, n_pages)
    rows = sum(counts)
    t = table_of(1000, pairs, sections, interleaved)
    places = np.concatenate([np.arange(n - c, n) for n, c in zip(lens, counts)])[:, None]
    given = t.axes > 1 or strided
    pos = rng.integers(0, 1000, (rows, t.axes)) if given else places
    k, v = rows_of(rng, rows, heads, d), rows_of(rng, rows, heads, d)
    q = rows_of(rng, rows, q_heads, d) if q_heads else None
    cs = t.cos_sin.cpu().numpy()
    turned = P.rope_steps(k.float().numpy(), cs, pos, axis_of(t), interleaved)
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    P.append(pool, turned, v.double().numpy(), table, lens, counts)
    kk, vv, qq = k.cuda(), v.cuda(), None if q is None else q.cuda()
    if strided:   # one fused projection, heads apart
        wide = torch.zeros(rows, q_heads + 2 * heads + 1, d, dtype=torch.bfloat16, device="cuda")
        wide[:, 1:heads + 1], wide[:, heads + 1:2 * heads + 1] = kk, vv
        kk, vv = wide[:, 1:heads + 1], wide[:, heads + 1:2 * heads + 1]
        if q is not None:
            wide[:, 2 * heads + 1:] = qq
            qq = wide[:, 2 * heads + 1:]
    one = all(n == 1 for n in counts)
    for off in ([offsets_of(counts)] + ([None] if one else [])):
        cache = cache_of(codes, exps)
        got = kvq.pages_append_rope(cache, t, kk, vv, dev(table), dev(lens), off, positions=dev(pos) if given else None, q=qq)
        clean()
        for kv, (c, s) in enumerate(((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale))):
            assert np.array_equal(exps_of(s)[0], pool.exp[kv])
            assert np.array_equal(P.VALUES[codes_of(c)[0]], pool.val[kv])
        if q is None:
            assert got is None
        else:
            want = P.rope_steps(q.float().numpy(), cs, pos, axis_of(t), interleaved)
            assert np.array_equal(bits(got), bits(torch.from_numpy(want).bfloat16()))
    if q is not None:   # in place
        cache = cache_of(codes, exps)
        assert kvq.pages_append_rope(cache, t, kk, vv, dev(table), dev(lens), offsets_of(counts),
                                     positions=dev(pos) if given else None, q=qq, q_out=qq) is qq
        clean()
        assert torch.equal(qq, got)


def test_append_of_unturned_rows_is_the_plain_append():
    """At position 0 every bit is that of pages_append."""
    rng = np.random.default_rng(5)
    lens, counts = [70, 33], [40, 33]
    codes, exps = random_pool(1, 2, 12, 3, 16, 128)
    t = table_of(4, 64, [22, 21, 21], True)
    k, v = rows_of(rng, 73, 3, 128).cuda(), rows_of(rng, 73, 3, 128).cuda()
    table = dev(make_table(rng, lens, 16, 12))
    a, b = cache_of(codes, exps), cache_of(codes, exps)
    kvq.pages_append(a, k, v, table, dev(lens), offsets_of(counts), layer=1)
    zero = torch.zeros(73, 3, dtype=torch.int32, device="cuda")
    kvq.pages_append_rope(b, t, k, v, table, dev(lens), offsets_of(counts), positions=zero, layer=1)
    clean()
    for x, y in ((a.k_codes, b.k_codes), (a.v_codes, b.v_codes)):
        assert np.array_equal(P.VALUES[codes_of(x)], P.VALUES[codes_of(y)])
    assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)


@pytest.mark.parametrize("given", [False, True])
def test_rows_outside_the_offsets_are_left(given):
    rng = np.random.default_rng(0)
    codes, exps = random_pool(1, 1, 6, 2, 16, 64)
    cache, t = cache_of(codes, exps), table_of(40, 32, None, False)
    k = rows_of(rng, 20, 2, 64)
    k[:3], k[13:] = float("nan"), float("nan")
    q = rows_of(rng, 20, 4, 64).cuda()
    out = torch.full_like(q, 9.0)
    table = make_table(rng, [30], 16, 6)
    pos = np.full((20, 1), 99)                                    # outside the table where no row is read
    pos[3:13, 0] = np.arange(20, 30)
    kvq.pages_append_rope(cache, t, k.cuda(), k.cuda(), dev(table), dev([30]), dev([3, 13]),
                          positions=dev(pos) if given else None, q=q, q_out=out)
    clean()
    cs = t.cos_sin.cpu().numpy()
    pool = P.Pool([c[0].numpy() for c in codes], [e[0] for e in exps])
    P.append(pool, P.rope_steps(k[3:13].float().numpy(), cs, pos[3:13], [0] * 32, False), k[3:13].double().numpy(), table, [30], [10])
    for kv, c in enumerate((cache.k_codes, cache.v_codes)):
        assert np.array_equal(P.VALUES[codes_of(c)[0]], pool.val[kv])
    assert (out[:3] == 9).all() and (out[13:] == 9).all()
    want = P.rope_steps(q[3:13].float().cpu().numpy(), cs, pos[3:13], [0] * 32, False)
    assert np.array_equal(bits(out[3:13]), bits(torch.from_numpy(want).bfloat16()))


def test_append_records_what_it_cannot_place():
    rng = np.random.default_rng(0)
    codes, exps = random_pool(1, 1, 4, 1, 16, 64)
    t = table_of(20, 32, None, False)
    k = rows_of(rng, 1, 1, 64).cuda()
    cache = cache_of(codes, exps)
    kvq.pages_append_rope(cache, t, k, k, dev([[0, 1]]), dev([25]))             # place 24: beyond the rotations
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_ERR_POSITION
    cache = cache_of(codes, exps)
    kvq.pages_append_rope(cache, t, k, k, dev([[7, 9]]), dev([1]))              # no such page
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_ERR_PAGE
    assert all(np.array_equal(codes_of(c), w.numpy()) for c, w in zip((cache.k_codes, cache.v_codes), codes))
    k[0, 0, 40] = float("inf")
    kvq.pages_append_rope(cache, t, k, torch.ones_like(k), dev([[0, 1]]), dev([3]))
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_ERR_RANGE and exps_of(cache.k_scale)[0, 0, 0] == 60


def test_streams_and_graphs():
    """On a stream of its own, and captured: a replay follows lengths, positions
    and rows that changed."""
    rng = np.random.default_rng(8)
    codes, exps = random_pool(2, 1, 9, 2, 16, 64)
    t = table_of(100, 32, None, False)
    k, v, q = (rows_of(rng, 3, h, 64).cuda() for h in (2, 2, 4))
    table, lens = dev(np.arange(9).reshape(3, 3)), dev([5, 17, 33])
    want = cache_of(codes, exps)
    want_q = kvq.pages_append_rope(want, t, k, v, table, lens, q=q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = cache_of(codes, exps)
    torch.cuda.synchronize()
    got_q = kvq.pages_append_rope(got, t, k, v, table, lens, q=q, stream=side)
    turned = kvq.rope(t, q, lens, stream=side)
    side.synchronize()
    clean()
    assert torch.equal(got_q, want_q) and torch.equal(got.k_codes.view(torch.uint8), want.k_codes.view(torch.uint8))
    assert torch.equal(turned, kvq.rope(t, q, lens))
    cache = cache_of(codes, exps)
    k0, lens0 = k.clone(), lens.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kvq.pages_append_rope(cache, t, k0, v, table, lens0, q=q)
        both = kvq.rope(t, q, lens0, k=k0)
    fresh = cache_of(codes, exps)
    for a, b in ((cache.k_codes, fresh.k_codes), (cache.v_codes, fresh.v_codes)):
        a.view(torch.uint8).copy_(b.view(torch.uint8))
    cache.k_scale.copy_(fresh.k_scale)
    cache.v_scale.copy_(fresh.v_scale)
    k0.copy_(k * 2)
    lens0.copy_(lens + 1)
    graph.replay()
    clean()
    want_q = kvq.pages_append_rope(fresh, t, k * 2, v, table, lens + 1, q=q)
    assert torch.equal(out, want_q) and torch.equal(cache.k_codes.view(torch.uint8), fresh.k_codes.view(torch.uint8))
    assert torch.equal(cache.k_scale, fresh.k_scale)
    eager = kvq.rope(t, q, lens + 1, k=k * 2)
    assert torch.equal(both[0], eager[0]) and torch.equal(both[1], eager[1])


def test_rows_beyond_32_bit_offsets():
    """Rows whose elements stand past 2^31 of their tensor's start."""
    t = table_of(16, 64, None, False)
    big = torch.empty(2 ** 24 + 40, 1, 136, dtype=torch.bfloat16, device="cuda")[..., :128]
    x = rows_of(np.random.default_rng(0), 40, 1, 128).cuda()
    big[-40:] = x
    pos = torch.zeros(big.shape[0], 1, dtype=torch.int32, device="cuda")
    pos[-40:, 0] = torch.arange(40, device="cuda") % 16
    kvq.rope(t, big, pos, q_out=big)
    clean()
    assert torch.equal(big[-40:], kvq.rope(t, x, pos[-40:].contiguous()))


def test_append_then_attention_over_rotated_keys():
    """A layer's step as it is used: queries and keys turned on the way, then
    attention; the scores depend on distances alone, so a sequence whose
    positions all start later gives the same output."""
    from tests.paged_common import check_attention
    rng = np.random.default_rng(11)
    lens, counts = [90, 37], [90, 37]
    t = table_of(400, 64, None, False)
    q, k, v = (rows_of(rng, 127, h, 128) for h in (4, 2, 2))
    table = make_table(rng, lens, 16, 10)
    places = np.concatenate([np.arange(n) for n in lens])
    cs = t.cos_sin.cpu().numpy()
    for start in (0, 250):
        cache = kvq.PagedCache.zeros(1, 10, 2, 16, 128)
        pos = (places + start)[:, None]
        turned = kvq.pages_append_rope(cache, t, k.cuda(), v.cuda(), dev(table), dev(lens), offsets_of(counts),
                                       positions=dev(pos) if start else None, q=q.cuda())
        got = kvq.paged_attention(cache, turned, dev(table), dev(lens), offsets_of(counts), max_q=90, with_lse=True)
        clean()
        pool = P.Pool([np.zeros((10, 2, 16, 128), np.uint8)] * 2, [np.zeros((10, 2), int)] * 2)
        P.append(pool, P.rope_steps(k.float().numpy(), cs, pos, [0] * 64, False), v.double().numpy(), table, lens, counts)
        qt = torch.from_numpy(P.rope_steps(q.float().numpy(), cs, pos, [0] * 64, False)).bfloat16()
        ref = P.attention(pool, qt.double().numpy(), table, lens, counts, 128 ** -0.5, True, 0)
        check_attention(got, ref, 128, 90, what=str(start))
