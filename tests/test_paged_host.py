"""The paged 8-bit cache on the host (no GPU): its oracle against hand-worked
values, the refusals of the C ABI and of the binding, the mirrored structs."""
import ctypes
import os
import shutil
import subprocess
import tempfile

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from quantized_kv_cache_quantize_gb300 import kvq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 0x10000   # aligned, never dereferenced: every call below is refused or a no-op


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kvq.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return kvq.lib()


# ---- the oracle ----

def test_e4m3_values_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(P.VALUES, want, equal_nan=True)


def test_e4m3_round_by_hand_and_by_search():
    for x, want in ((0.0, 0.0), (1.0, 1.0), (1.0625, 1.0), (1.1875, 1.25), (448.0, 448.0), (463.0, 448.0),
                    (500.0, 448.0), (-17.0, -16.0), (-19.0, -20.0), (2.0 ** -10, 0.0), (1.5 * 2.0 ** -9, 2.0 ** -8),
                    (2.0 ** -9, 2.0 ** -9), (248.0, 256.0), (232.0, 224.0)):
        assert P.e4m3_round(x) == want, x
    rng = np.random.default_rng(0)
    x = rng.standard_normal(4000) * np.exp2(rng.integers(-12, 8, 4000))
    grid = np.unique(P.VALUES[~np.isnan(P.VALUES)])
    near = np.abs(grid[None] - x[:, None]).min(1)
    assert np.array_equal(np.abs(P.e4m3_round(x) - x), near)
    assert np.array_equal(P.VALUES[P.e4m3_code(P.e4m3_round(x))], P.e4m3_round(x))


def test_scale_exponent_by_hand():
    for amax, e in ((0.0, -60), (448.0, 0), (448.0001, 1), (449.0, 1), (224.0, -1), (1.75, -8), (1.76, -7), (1.0, -8),
                    (1e-30, -60), (1e30, 60)):
        assert P.scale_exponent(amax) == e, amax


def test_growing_scale_keeps_normal_codes():
    """Tokens appended one by one end at the codes of one append of all, but
    for values that become E4M3 subnormals."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((8, 1, 64)) * np.exp2(rng.integers(-2, 4, (8, 1, 1)))
    pools = [P.Pool([np.zeros((1, 1, 16, 64), np.uint8)] * 2, [np.zeros((1, 1), int)] * 2) for _ in range(2)]
    P.append(pools[0], x, x, [[0]], [8], [8])
    for i in range(8):
        P.append(pools[1], x[i:i + 1], x[i:i + 1], [[0]], [i + 1], [1])
    a, b = pools[0].val[0][0, 0, :8], pools[1].val[0][0, 0, :8]
    assert pools[0].exp[0][0, 0] == pools[1].exp[0][0, 0]
    normal = np.abs(a) >= 2.0 ** -6
    assert normal.mean() > 0.9 and np.array_equal(a[normal], b[normal])


def test_compact_oracle_by_hand():
    t, n, moves = P.compact([[5, 2, -1], [9, 5, 0]], 12)
    assert n == 4 and moves == [(5, 1), (9, 3)]
    assert t.tolist() == [[1, 2, -1], [3, 1, 0]]


# ---- the C ABI ----

def _pages(**kw):
    c = kvq.PagesStruct()
    c.layers, c.n_pages, c.kv_heads, c.head_dim, c.page_tokens = 2, 10, 4, 128, 16
    c.k_codes = c.v_codes = c.k_scale = c.v_scale = PTR
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _seqs(**kw):
    s = kvq.SequencesStruct()
    s.batch, s.width, s.table_stride, s.rows = 3, 5, 5, 3
    s.table = s.kv_lens = PTR
    s.offsets = None
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_pages_bytes(lib):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.kvq_pages_bytes(ctypes.byref(_pages()), ctypes.byref(a), ctypes.byref(b)) == 0
    assert a.value == 2 * 10 * 4 * 16 * 128 and b.value == 2 * 10 * 4 * 2
    big = _pages(layers=64, n_pages=1 << 20, kv_heads=8, page_tokens=128)
    assert lib.kvq_pages_bytes(ctypes.byref(big), ctypes.byref(a), None) == 0
    assert a.value == 64 * (1 << 20) * 8 * 128 * 128


GEOMETRY = [("head_dim", 96, kvq.KVQ_ERR_UNSUPPORTED), ("page_tokens", 8, kvq.KVQ_ERR_UNSUPPORTED),
            ("page_tokens", 48, kvq.KVQ_ERR_UNSUPPORTED), ("layers", 0, kvq.KVQ_ERR_INVALID_ARG),
            ("n_pages", 0, kvq.KVQ_ERR_INVALID_ARG), ("kv_heads", 0, kvq.KVQ_ERR_INVALID_ARG),
            ("n_pages", 1 << 30, kvq.KVQ_ERR_INVALID_ARG)]
BUFFERS = [("k_codes", 0, kvq.KVQ_ERR_INVALID_ARG), ("v_scale", 0, kvq.KVQ_ERR_INVALID_ARG),
           ("v_codes", PTR + 8, kvq.KVQ_ERR_ALIGNMENT), ("k_scale", PTR + 1, kvq.KVQ_ERR_ALIGNMENT)]


def _append(lib, c=None, s=None, layer=0, k=PTR, v=PTR, ks=(512, 128), vs=(512, 128)):
    c, s = c or _pages(), s or _seqs()
    return lib.kvq_pages_append(ctypes.byref(c), layer, k, *ks, v, *vs, ctypes.byref(s), None)


def _attend(lib, c=None, s=None, layer=0, q=PTR, qs=(1024, 128), heads=8, max_q=1, scale=0.1, window=0, ws=PTR,
            ws_bytes=1 << 40, out=PTR, lse=None):
    c, s = c or _pages(), s or _seqs()
    return lib.kvq_paged_attention(ctypes.byref(c), layer, q, *qs, heads, ctypes.byref(s), max_q, scale, 1, window, ws,
                                   ws_bytes, out, lse, None)


def _compact(lib, c=None, table=PTR, batch=3, width=5, stride=5, out=PTR, out_stride=5, n=PTR, ws=PTR, ws_bytes=1 << 30):
    c = c or _pages()
    return lib.kvq_pages_compact(ctypes.byref(c), table, batch, width, stride, out, out_stride, n, ws, ws_bytes, None)


def _copy(lib, src, dst, c=None, n=None):
    a, b = (np.asarray(x, np.int32) for x in (src, dst))
    c = c or _pages()
    return lib.kvq_pages_copy(ctypes.byref(c), a.ctypes.data, b.ctypes.data, len(a) if n is None else n, None)


@pytest.mark.parametrize("field,value,status", GEOMETRY + BUFFERS)
def test_bad_pool(lib, field, value, status):
    c = _pages(**{field: value})
    if (field, value, status) in GEOMETRY:
        assert lib.kvq_pages_bytes(ctypes.byref(c), None, None) == status
        assert lib.kvq_paged_workspace_bytes(ctypes.byref(c), 8, 1, 1, 1, 1) == 0
        assert lib.kvq_pages_compact_workspace_bytes(ctypes.byref(c)) == 0
    assert _append(lib, c) == status
    assert _attend(lib, c) == status
    assert _compact(lib, c) == status
    assert _copy(lib, [1], [2], c) == status


@pytest.mark.parametrize("fields,status", [
    (dict(batch=-1), 1), (dict(width=-1), 1), (dict(rows=-1), 1), (dict(rows=2), 1), (dict(kv_lens=None), 1),
    (dict(table=None), 1), (dict(table_stride=4), 1), (dict(table=PTR + 2), 6), (dict(kv_lens=PTR + 1), 6),
    (dict(offsets=PTR + 2), 6), (dict(batch=0, rows=4, offsets=PTR), 1)])
def test_bad_sequences(lib, fields, status):
    s = _seqs(**fields)
    assert _append(lib, s=s) == status
    assert _attend(lib, s=s) == status


def test_append_refusals(lib):
    assert _append(lib, layer=2) == 1 and _append(lib, layer=-1) == 1
    assert _append(lib, k=None) == 1 and _append(lib, v=None) == 1
    assert _append(lib, k=PTR + 8) == 6 and _append(lib, v=PTR + 2) == 6
    assert _append(lib, ks=(4, 128)) == 6 and _append(lib, vs=(512, -128)) == 6
    assert lib.kvq_pages_append(None, 0, PTR, 512, 128, PTR, 512, 128, ctypes.byref(_seqs()), None) == 1
    assert lib.kvq_pages_append(ctypes.byref(_pages()), 0, PTR, 512, 128, PTR, 512, 128, None, None) == 1
    assert _append(lib, s=_seqs(rows=0, batch=0)) == 0          # nothing to append
    assert _append(lib, c=_pages(n_pages=1, kv_heads=1 << 10),
                   s=_seqs(rows=1 << 30, batch=2, offsets=PTR)) == kvq.KVQ_ERR_TOO_LARGE


def test_attention_refusals(lib):
    assert _attend(lib, layer=2) == 1
    assert _attend(lib, heads=6) == 1 and _attend(lib, heads=0) == 1
    assert _attend(lib, scale=float("nan")) == 1 and _attend(lib, scale=0.0) == 1
    assert _attend(lib, window=-1) == 1 and _attend(lib, max_q=0) == 1
    assert _attend(lib, q=None) == 1 and _attend(lib, out=None) == 1
    wide = _seqs(width=1 << 16, table_stride=1 << 16)          # long sequences: parts go through the workspace
    need = lib.kvq_paged_workspace_bytes(ctypes.byref(_pages()), 8, 3, 1 << 16, 3, 1)
    assert need > 16
    assert _attend(lib, s=wide, ws=None) == 1 and _attend(lib, s=wide, ws_bytes=need - 1) == 1
    assert _attend(lib, s=_seqs(width=1 << 27, table_stride=1 << 27)) == kvq.KVQ_ERR_TOO_LARGE
    assert _append(lib, s=_seqs(width=1 << 27, table_stride=1 << 27)) == kvq.KVQ_ERR_TOO_LARGE
    assert _attend(lib, q=PTR + 2) == 6 and _attend(lib, out=PTR + 2) == 6 and _attend(lib, lse=PTR + 2) == 6
    assert _attend(lib, ws=PTR + 8) == 6 and _attend(lib, qs=(1024, 12)) == 6
    assert _attend(lib, s=_seqs(rows=0, batch=0)) == 0
    c = _pages()
    assert lib.kvq_paged_workspace_bytes(ctypes.byref(c), 6, 1, 1, 1, 1) == 0


def test_copy_refusals(lib):
    assert _copy(lib, [], []) == 0
    assert _copy(lib, [1], [2], n=-1) == 1
    assert lib.kvq_pages_copy(ctypes.byref(_pages()), None, None, 1, None) == 1
    for src, dst in (([0], [10]), ([10], [0]), ([-1], [0]), ([0], [-1]),       # outside the pool
                     ([0, 1], [2, 2]),                                         # a destination twice
                     ([0, 1], [1, 2]), ([3, 0], [0, 4]), ([3], [3])):          # a destination that is read
        assert _copy(lib, src, dst) == 1, (src, dst)


def test_compact_refusals(lib):
    assert _compact(lib, _pages(n_pages=(1 << 20) + 1)) == kvq.KVQ_ERR_TOO_LARGE
    assert _compact(lib, n=None) == 1 and _compact(lib, ws=None) == 1 and _compact(lib, table=None) == 1
    assert _compact(lib, out=None) == 1 and _compact(lib, stride=4) == 1 and _compact(lib, out_stride=4) == 1
    assert _compact(lib, out_stride=6) == 1                      # in place, but at another stride
    assert _compact(lib, batch=-1) == 1 and _compact(lib, width=-1) == 1
    assert _compact(lib, table=PTR + 2) == 6 and _compact(lib, n=PTR + 1) == 6 and _compact(lib, ws=PTR + 4) == 6
    assert _compact(lib, ws_bytes=kvq.lib().kvq_pages_compact_workspace_bytes(ctypes.byref(_pages())) - 1) == 1


def test_page_status(lib):
    assert kvq.KVQ_ERR_PAGE == 10 and "paged" in kvq.status_string(kvq.KVQ_ERR_PAGE)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
@pytest.mark.parametrize("cls,name", [(kvq.PagesStruct, "kvq_pages"), (kvq.SequencesStruct, "kvq_sequences")])
def test_structs_mirror_the_header(cls, name):
    fields = [f[0] for f in cls._fields_]
    prog = ["#include <stddef.h>", "#include <stdio.h>", '#include "kvq.h"', "int main(void) {",
            f'  printf("%zu\\n", sizeof({name}));']
    prog += [f'  printf("%zu\\n", offsetof({name}, {f}));' for f in fields] + ["  return 0;", "}"]
    with tempfile.TemporaryDirectory() as tmp:
        src, exe = os.path.join(tmp, "layout.c"), os.path.join(tmp, "layout")
        with open(src, "w") as f:
            f.write("\n".join(prog) + "\n")
        subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", exe, src])
        got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got[0] == ctypes.sizeof(cls)
    assert got[1:] == [getattr(cls, f).offset for f in fields]


# ---- the binding ----

def test_binding_refusals(lib):
    f8, bf = torch.float8_e4m3fn, torch.bfloat16
    codes = torch.zeros(2, 10, 4, 16, 64, dtype=torch.uint8).view(f8)
    scale = torch.ones(2, 10, 4, dtype=bf)
    cache = kvq.PagedCache(codes, codes.clone(), scale, scale.clone())
    assert (cache.layers, cache.n_pages, cache.kv_heads, cache.page_tokens, cache.head_dim) == (2, 10, 4, 16, 64)
    for bad in ((codes[0], codes, scale, scale), (codes, codes[:1], scale, scale),
                (codes, codes.view(torch.uint8), scale, scale), (codes, codes, scale.float(), scale),
                (codes, codes, scale, scale[:1]), (codes, codes.transpose(1, 2), scale, scale)):
        with pytest.raises(ValueError):
            kvq.PagedCache(*bad)
    with pytest.raises(kvq.KVQError, match="unsupported"):
        wide = torch.zeros(1, 2, 2, 16, 96, dtype=torch.uint8).view(f8)
        kvq.PagedCache(wide, wide, torch.ones(1, 2, 2, dtype=bf), torch.ones(1, 2, 2, dtype=bf))
    x = torch.zeros(3, 4, 64, dtype=bf)
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    for bad in (torch.zeros(3, 4, 128, dtype=bf), torch.zeros(3, 256, dtype=bf), x):     # x: right shape, on the CPU
        with pytest.raises(ValueError):
            kvq.pages_append(cache, bad, bad, table, lens)
        with pytest.raises(ValueError):
            kvq.paged_attention(cache, bad, table, lens)
    with pytest.raises(ValueError, match="CUDA int32"):
        kvq.pages_compact(cache, table)
    for src, dst in (([1], [2, 3]), ([0.5], [1]), ([1 << 40], [1]), (torch.tensor([-1]), [1]),
                     (torch.ones(1, 1, dtype=torch.int32), [1])):
        with pytest.raises(ValueError, match="src|outside|list|dst"):
            kvq.pages_copy(cache, src, dst)
    with pytest.raises(ValueError, match="not a CUDA device"):
        kvq.pages_copy(cache, [1], [2])


def test_arguments_beyond_32_bits(lib):
    """Refused, not cut: 2^32 + 5 would arrive as a window of 5."""
    codes = torch.zeros(1, 2, 1, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    cache = kvq.PagedCache(codes, codes.clone(), *[torch.ones(1, 2, 1, dtype=torch.bfloat16) for _ in range(2)])
    x, table, lens = torch.zeros(1, 1, 64), torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for kw in (dict(window=(1 << 32) + 5), dict(layer=1 << 32), dict(max_q=(1 << 33) + 1)):
        with pytest.raises(ValueError, match="beyond 32 bits"):
            kvq.paged_attention(cache, x, table, lens, **kw)
    with pytest.raises(ValueError, match="beyond 32 bits"):
        kvq.pages_append(cache, x, x, table, lens, layer=-(1 << 32))
    assert _attend(lib, s=_seqs(rows=(1 << 30) + 1, offsets=PTR)) == kvq.KVQ_ERR_TOO_LARGE
    assert _append(lib, s=_seqs(rows=(1 << 30) + 1, offsets=PTR)) == kvq.KVQ_ERR_TOO_LARGE
