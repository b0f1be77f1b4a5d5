"""Rotary positions on the host (no GPU): the oracle, the refusals of the C ABI
and of the binding, the mirrored structs."""
import ctypes
import math
import os
import shutil

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from quantized_kv_cache_quantize_gb300 import kvq
from tests.test_paged_host import PTR, _pages, _seqs, test_structs_mirror_the_header as mirror


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kvq.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return kvq.lib()


# ---- the oracle ----

@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_by_hand(interleaved):
    """A quarter turn of pair 0 takes (1, 2) to (-2, 1); the rest stays."""
    x = np.zeros((1, 1, 8))
    at = (0, 1) if interleaved else (0, 2)
    x[0, 0, at[0]], x[0, 0, at[1]], x[0, 0, 7] = 1, 2, 5
    y = P.rope(x, [[1]], [math.pi / 2, 0.0], [0, 0], interleaved)
    want = x.copy()
    want[0, 0, at[0]], want[0, 0, at[1]] = -2, 1
    assert np.allclose(y, want, atol=1e-15)
    assert np.allclose(P.rope(y, [[1]], [math.pi / 2, 0.0], [0, 0], interleaved, inverse=True), x, atol=1e-15)


def test_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 64))
    f, axis = kvq.rope_frequencies(32, sections=[16, 8, 8]), [0] * 16 + [1] * 8 + [2] * 8
    dots = [float((P.rope(q[None], [a], f, axis, False) * P.rope(k[None], [b], f, axis, False)).sum())
            for a, b in (((5, 2, 9), (1, 2, 3)), ((105, 42, 19), (101, 42, 13)))]
    assert abs(dots[0] - dots[1]) < 1e-12


@pytest.mark.parametrize("interleaved", [False, True])
def test_steps_agree_with_the_definition(interleaved):
    rng = np.random.default_rng(1)
    x, pos, axis = rng.standard_normal((9, 2, 64)), rng.integers(0, 50, (9, 2)), [0, 1] * 8
    f = kvq.rope_frequencies(16)
    angle = np.arange(50)[:, None] * np.array(f)
    cs = np.stack([np.cos(angle), np.sin(angle)], -1).astype(np.float32)
    for inverse in (False, True):
        got, want = P.rope_steps(x.astype(np.float32), cs, pos, axis, interleaved, inverse), P.rope(x.astype(np.float32), pos, f, axis, interleaved, inverse)
        # two products, one sum and the table's entries: 2^-24 each, of |x0| + |x1| at most
        assert np.abs(got - want).max() <= 4 * 2.0 ** -24 * 2 * np.abs(x).max()


def test_frequencies():
    assert kvq.rope_frequencies(4, 100.0) == [1.0, 100.0 ** -0.25, 0.1, 100.0 ** -0.75]
    assert kvq.rope_frequencies(3, 16.0, [2, 1]) == [1.0, 0.25, 1.0]
    with pytest.raises(ValueError):
        kvq.rope_frequencies(4, sections=[2, 1])


# ---- the C ABI ----

def _table(**kw):
    t = kvq.RopeTableStruct()
    t.cos_sin, t.n_positions, t.pairs, t.axes = PTR, 100, 32, 1
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _rope(lib, t=None, pos=PTR, batch=1, rows=3, d=128, n=1, **kw):
    a = (kvq.RopeTensorStruct * 2)()
    for x in a:
        x.x = x.y = PTR
        x.x_row_stride = x.y_row_stride = 1024
        x.x_head_stride = x.y_head_stride = 128
        x.heads = 8
        for k, v in kw.items():
            setattr(x, k, v)
    t = t or _table()
    return lib.kvq_rope(ctypes.byref(t), pos, 0, 1, 0, batch, rows, d, 0, a, n, None)


def _append(lib, t=None, c=None, s=None, layer=0, pos=None, k=PTR, v=PTR, ks=(512, 128), vs=(512, 128), q=PTR,
            qs=(1024, 128), heads=8, out=PTR, outs=(1024, 128)):
    c, s, t = c or _pages(), s or _seqs(), t or _table()
    return lib.kvq_pages_append_rope(ctypes.byref(c), layer, ctypes.byref(t), pos, 1, k, *ks, v, *vs, q, *qs, heads, out,
                                     *outs, ctypes.byref(s), None)


BAD_TABLES = [(dict(cos_sin=None), 1), (dict(cos_sin=PTR + 8), 6), (dict(n_positions=0), 1), (dict(pairs=0), 1),
              (dict(pairs=12), 1), (dict(pairs=72), 1), (dict(axes=0), 1), (dict(axes=5), 1)]


@pytest.mark.parametrize("fields,status", BAD_TABLES)
def test_bad_table(lib, fields, status):
    t = _table(**fields)
    assert _rope(lib, t) == status
    assert _append(lib, t) == status
    f = (ctypes.c_double * 64)()
    assert lib.kvq_rope_fill(ctypes.byref(t), f, 1.0, None) == status


def test_table_against_the_head_and_its_axes(lib):
    t = _table()
    t.axis[31] = 1                                               # an axis that no position has
    assert _rope(lib, t) == 1 and _append(lib, t) == 1
    wide = _table(pairs=40)
    assert _rope(lib, wide, d=64) == 1                           # 80 channels of 64
    assert _append(lib, wide, c=_pages(head_dim=64)) == 1
    assert _rope(lib, d=96) == kvq.KVQ_ERR_UNSUPPORTED


def test_fill_refusals(lib):
    f = (ctypes.c_double * 64)()
    assert lib.kvq_rope_fill(ctypes.byref(_table()), None, 1.0, None) == 1
    assert lib.kvq_rope_fill(ctypes.byref(_table()), f, math.nan, None) == 1
    f[31] = math.inf
    assert lib.kvq_rope_fill(ctypes.byref(_table()), f, 1.0, None) == 1
    assert lib.kvq_rope_fill(None, f, 1.0, None) == 1


def test_rope_refusals(lib):
    assert _rope(lib, n=0) == 1 and _rope(lib, n=3) == 1 and _rope(lib, batch=-1) == 1 and _rope(lib, rows=-1) == 1
    assert _rope(lib, pos=None) == 1 and _rope(lib, pos=PTR + 2) == 6
    assert _rope(lib, x=None) == 1 and _rope(lib, y=None, n=2) == 1 and _rope(lib, heads=-1) == 1
    assert _rope(lib, x=PTR + 8) == 6 and _rope(lib, y=PTR + 2) == 6
    for field in ("x_batch_stride", "x_row_stride", "x_head_stride", "y_batch_stride", "y_row_stride", "y_head_stride"):
        assert _rope(lib, **{field: 12}) == 6 and _rope(lib, **{field: -8}) == 6
    assert _rope(lib, y_batch_stride=4096, batch=2) == 1         # in place, but other places
    assert _rope(lib, y_row_stride=4096) == 1 and _rope(lib, y_head_stride=4096) == 1
    assert _rope(lib, n=2) == 1                                  # one writes what the other writes
    assert _rope(lib, rows=0) == 0 and _rope(lib, batch=0) == 0 and _rope(lib, heads=0, x=None, y=None) == 0
    assert _rope(lib, batch=1 << 16, rows=1 << 16) == kvq.KVQ_ERR_TOO_LARGE
    assert _rope(lib, rows=1 << 30, heads=64) == kvq.KVQ_ERR_TOO_LARGE
    assert _rope(lib, rows=1, batch=1 << 30, heads=32) == kvq.KVQ_ERR_TOO_LARGE
    assert lib.kvq_rope(ctypes.byref(_table()), PTR, 0, 1, 0, 1, 1, 128, 0, None, 1, None) == 1


def test_append_refusals(lib):
    assert _append(lib, layer=2) == 1 and _append(lib, k=None) == 1 and _append(lib, v=None) == 1
    assert _append(lib, k=PTR + 8) == 6 and _append(lib, ks=(4, 128)) == 6
    assert _append(lib, q=None) == 1 and _append(lib, out=None) == 1 and _append(lib, heads=0) == 1
    assert _append(lib, heads=-1) == 1 and _append(lib, q=None, heads=0) == 1
    assert _append(lib, q=PTR + 8) == 6 and _append(lib, out=PTR + 8) == 6 and _append(lib, pos=PTR + 2) == 6
    assert _append(lib, qs=(12, 128)) == 6 and _append(lib, outs=(1024, -128)) == 6
    assert _append(lib, _table(axes=3)) == 1                     # several axes need positions
    apart = dict(k=PTR + (1 << 20), v=PTR + (1 << 21))
    assert _append(lib, outs=(2048, 128), **apart) == 1 and _append(lib, outs=(1024, 256), **apart) == 1
    assert _append(lib, k=PTR + (1 << 20)) == 1 and _append(lib, v=PTR + (1 << 21)) == 1   # queries over the values, the keys
    assert _append(lib, s=_seqs(rows=0, batch=0)) == 0
    assert _append(lib, s=_seqs(rows=1 << 30, batch=2, offsets=PTR), heads=64, qs=(8192, 128), outs=(8192, 128)) == kvq.KVQ_ERR_TOO_LARGE
    for fields, status in ((dict(batch=-1), 1), (dict(table=None), 1), (dict(table_stride=4), 1), (dict(kv_lens=PTR + 1), 6)):
        assert _append(lib, s=_seqs(**fields)) == status
    for fields, status in ((dict(head_dim=96), 2), (dict(page_tokens=8), 2), (dict(k_codes=0), 1)):
        assert _append(lib, c=_pages(**fields)) == status


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
@pytest.mark.parametrize("cls,name", [(kvq.RopeTableStruct, "kvq_rope_table"), (kvq.RopeTensorStruct, "kvq_rope_tensor")])
def test_structs_mirror_the_header(cls, name):
    mirror(cls, name)


def test_position_status(lib):
    assert kvq.KVQ_ERR_POSITION == 11 and "position" in kvq.status_string(kvq.KVQ_ERR_POSITION)


# ---- the binding ----

def test_table_of_the_binding(lib):
    cs = torch.zeros(10, 32, 2)
    t = kvq.RopeTable(cs, [16, 8, 8], True)
    assert (t.n_positions, t.pairs, t.axes, t.interleaved) == (10, 32, 3, True)
    assert list(t.struct.axis)[:32] == [0] * 16 + [1] * 8 + [2] * 8
    t = kvq.RopeTable(cs, axis=[0, 1] * 16)
    assert t.axes == 2 and list(t.struct.axis)[:4] == [0, 1, 0, 1]
    for bad in (cs[0], cs.double(), torch.zeros(10, 32, 3), torch.zeros(10, 2, 32).transpose(1, 2), torch.zeros(10, 12, 2),
                torch.zeros(10, 72, 2), torch.zeros(0, 32, 2)):
        with pytest.raises(ValueError):
            kvq.RopeTable(bad)
    for kw in (dict(sections=[16, 8]), dict(sections=[40, -8]), dict(sections=[8, 8, 8, 4, 4]), dict(axis=[0] * 31),
               dict(axis=[4] * 32), dict(axis=[-1] * 32), dict(sections=[32], axis=[0] * 32)):
        with pytest.raises(ValueError):
            kvq.RopeTable(cs, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.RopeTable.build(10, kvq.rope_frequencies(32), device="cpu")


def test_binding_refuses_host_tensors(lib):
    t = kvq.RopeTable(torch.zeros(10, 32, 2))
    x, pos = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for bad in (x, x.float(), x[0], torch.zeros(1, 1, 3, 4, 64, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            kvq.rope(t, bad, pos)
    codes = torch.zeros(1, 10, 4, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    cache = kvq.PagedCache(codes, codes.clone(), *[torch.ones(1, 10, 4, dtype=torch.bfloat16) for _ in range(2)])
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        kvq.pages_append_rope(cache, t, x, x, table, lens)
    with pytest.raises(ValueError, match="beyond 32 bits"):
        kvq.pages_append_rope(cache, t, x, x, table, lens, layer=1 << 32)


def test_packed_tensors_are_the_structure():
    """The binding packs kvq_rope_tensor and kvq_sequences by hand; ctypes' copies
    of them, which are checked against the header, have the same bytes."""
    a, b = tuple(range(1, 10)), tuple(range(11, 20))
    both = (kvq.RopeTensorStruct * 2)(kvq.RopeTensorStruct(*a), kvq.RopeTensorStruct(*b))
    assert kvq._packed_sequences(1, 2, 3, 4, 5, 6, 7) == bytes(kvq.SequencesStruct(1, 2, 3, 4, 5, 6, 7))
    assert kvq._rope_tensors(*a, *b) == bytes(both) and kvq._rope_tensor(*a) == bytes(both)[:ctypes.sizeof(kvq.RopeTensorStruct)]
