"""Shaped attention scores on the host (no GPU): the oracle against hand-worked
values, the refusals of the C ABI and of the binding, the mirrored struct."""
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


def _pool():
    """Four keys in one page, K one-hot times 2, 4, 6, 8 in channel 0, V the number of the key."""
    k, v = np.zeros((1, 1, 16, 64)), np.zeros((1, 1, 16, 64))
    k[0, 0, :4, 0], v[0, 0, :4] = [2, 4, 6, 8], np.arange(4)[:, None]
    codes = [P.e4m3_code(P.e4m3_round(x)) for x in (k, v)]
    return P.Pool(codes, [np.zeros((1, 1), int)] * 2)


def test_oracle_by_hand():
    q = np.zeros((2, 1, 64))
    q[:, 0, 0] = 0.5                                            # scores 1, 2, 3, 4; rows at positions 2 and 3
    args = (_pool(), q, [[0]], [4], [2], 1.0)
    o, lse = P.attention_scored(*args, True, 0, softcap=2.0)[:2]
    s = 2 * np.tanh(np.arange(1, 5) / 2)
    assert np.allclose(lse[:, 0], [np.log(np.exp(s[:3]).sum()), np.log(np.exp(s).sum())])
    assert np.allclose(o[1, 0, 0], (np.exp(s) * np.arange(4)).sum() / np.exp(s).sum())
    lse = P.attention_scored(*args, False, 0, slopes=[0.5])[1]
    s = np.arange(1, 5) - 0.5 * np.array([[2, 1, 0, 1], [3, 2, 1, 0]])
    assert np.allclose(lse[:, 0], np.log(np.exp(s).sum(1)))
    lse = P.attention_scored(*args, True, 0, prefix=[4])[1]
    assert np.allclose(lse[:, 0], np.log(np.exp(np.arange(1, 5)).sum()))
    lse = P.attention_scored(*args, True, 2, prefix=[4], ranges=[[0, 3], [3, 3]])[1]
    assert np.allclose(lse[0, 0], np.log(np.exp([2.0, 3.0]).sum())) and lse[1, 0] == -math.inf


def test_oracle_without_shapes_is_the_plain_one():
    rng = np.random.default_rng(0)
    q = rng.standard_normal((3, 2, 64))
    a, b = P.attention(_pool(), q, [[0]], [4], [3], 0.3, True, 2), P.attention_scored(_pool(), q, [[0]], [4], [3], 0.3, True, 2)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


# ---- the C ABI ----

def _attend(lib, c=None, s=None, layer=0, q=PTR, qs=(1024, 128), heads=8, max_q=1, scale=0.1, window=0, ws=PTR,
            ws_bytes=1 << 40, out=PTR, lse=None, **kw):
    x = kvq.ScoresStruct(5.0, None, None, None)
    for k, v in kw.items():
        setattr(x, k, v)
    c, s = c or _pages(), s or _seqs()
    return lib.kvq_paged_attention_scored(ctypes.byref(c), layer, q, *qs, heads, ctypes.byref(s), max_q, scale, 1, window,
                                          ctypes.byref(x), ws, ws_bytes, out, lse, None)


def test_refusals(lib):
    for cap in (-1.0, math.nan, math.inf, 2.0 ** -21, 2.0 ** 20 + 1):
        assert _attend(lib, softcap=cap) == 1, cap
    assert _attend(lib, slopes=PTR + 2) == 6 and _attend(lib, prefix=PTR + 1) == 6 and _attend(lib, ranges=PTR + 4) == 6
    assert _attend(lib, layer=2) == 1 and _attend(lib, heads=6) == 1 and _attend(lib, q=None) == 1
    assert _attend(lib, out=None) == 1 and _attend(lib, scale=math.nan) == 1 and _attend(lib, window=-1) == 1
    assert _attend(lib, max_q=0) == 1 and _attend(lib, qs=(1024, 12)) == 6 and _attend(lib, out=PTR + 2) == 6
    assert _attend(lib, s=_seqs(width=1 << 27, table_stride=1 << 27)) == kvq.KVQ_ERR_TOO_LARGE
    assert _attend(lib, c=_pages(head_dim=96)) == kvq.KVQ_ERR_UNSUPPORTED
    assert _attend(lib, s=_seqs(kv_lens=None)) == 1
    wide = _seqs(width=1 << 16, table_stride=1 << 16)
    need = lib.kvq_paged_workspace_bytes(ctypes.byref(_pages()), 8, 3, 1 << 16, 3, 1)
    assert need > 16
    assert _attend(lib, s=wide, ws=None) == 1 and _attend(lib, s=wide, ws_bytes=need - 1) == 1
    assert _attend(lib, s=_seqs(rows=0, batch=0)) == 0


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_struct_mirrors_the_header():
    mirror(kvq.ScoresStruct, "kvq_scores")


# ---- the binding ----

def test_binding_refusals(lib):
    codes = torch.zeros(1, 4, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    cache = kvq.PagedCache(codes, codes.clone(), *[torch.ones(1, 4, 2, dtype=torch.bfloat16) for _ in range(2)])
    ok = dict(softcap=0.0, slopes=None, prefix=None, ranges=None)
    assert kvq._scores(cache, 4, 2, 3, **ok) is None
    assert kvq._scores(cache, 4, 2, 3, **(ok | dict(softcap=None))) is None
    for cap in (-1.0, 1e-60, math.nan, math.inf, 2.0 ** 21):
        with pytest.raises(kvq.KVQError, match="softcap"):
            kvq._scores(cache, 4, 2, 3, **(ok | dict(softcap=cap)))
    assert kvq._scores(cache, 4, 2, 3, **(ok | dict(softcap=3.0))).softcap == 3.0
    good = dict(slopes=torch.ones(4), prefix=torch.ones(2, dtype=torch.int32), ranges=torch.zeros(3, 2, dtype=torch.int32))
    s = kvq._scores(cache, 4, 2, 3, 0.0, **good)
    assert (s.softcap, s.slopes, s.prefix, s.ranges) == (0.0, *[t.data_ptr() for t in good.values()])
    for name, bad in (("slopes", torch.ones(3)), ("slopes", torch.ones(4).half()), ("slopes", torch.ones(8)[::2]),
                      ("prefix", torch.ones(3, dtype=torch.int32)), ("prefix", torch.ones(2, dtype=torch.int64)),
                      ("ranges", torch.zeros(2, 3, dtype=torch.int32).T), ("ranges", torch.zeros(6, dtype=torch.int32))):
        with pytest.raises(ValueError, match=name):
            kvq._scores(cache, 4, 2, 3, **(ok | {name: bad}))


# ---- the polynomials of tanh ----

def _horner(c, x):
    """x times the polynomial in x^2, every step rounded to fp32 as the kernels do."""
    x = x.astype(np.float32)
    z = (x * x).astype(np.float32)
    p = np.full_like(z, c[-1])
    for k in c[-2::-1]:
        p = (p.astype(np.float64) * z + np.float64(k)).astype(np.float32)      # fused
    return p * x


@pytest.mark.parametrize("which,x_max,bound", [(0, 1.0, 2.0 ** -22), (1, 0.4, 2.0 ** -21.8)])
def test_tanh_polynomials(which, x_max, bound):
    """The constants in the kernels are the fit's, and near tanh to the bound that
    is stated beside them."""
    import re
    from quantized_kv_cache_quantize_gb300.csrc import tanh_fit
    fit = (tanh_fit.fit_coefficients(), tanh_fit.fit_coefficients(tanh_fit.LOW_TERMS, tanh_fit.LOW_X))[which].astype(np.float32)
    assert tanh_fit.LOW_X == 0.4
    src = open(os.path.join(os.path.dirname(tanh_fit.__file__), "kvq_scores.cuh")).read()
    have = {np.float32(v) for v in re.findall(r"-?\d\.\d+e[-+]\d+(?=f)", src)}
    assert {np.float32(c) for c in fit} <= have
    x = np.linspace(1e-4, x_max, 200001)
    assert np.abs(_horner(fit, x) / np.tanh(x.astype(np.float32).astype(np.float64)) - 1).max() <= bound
