"""The paged calls where their kernels change form or reach far: batches for
every split of the keys, rows that are not finite, pools beyond 4 GB, calls
captured apart and replayed together, and the build that checks its indices."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from quantized_kv_cache_quantize_gb300 import kvq
from tests.paged_common import check_attention, codes_of, dev, exps_of, offsets_of

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def clean():
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_OK


def fill(cache, seed):
    """Finite codes of every size and a scale of its own per page and head."""
    g = torch.Generator("cuda").manual_seed(seed)
    for t in (cache.k_codes, cache.v_codes):
        for layer in t.view(torch.uint8):
            for at in range(0, layer.shape[0], 4096):
                part = layer[at:at + 4096]
                part.copy_(torch.randint(0, 127, part.shape, generator=g, device="cuda", dtype=torch.uint8)
                           | torch.randint(0, 2, part.shape, generator=g, device="cuda", dtype=torch.uint8) << 7)
    for t in (cache.k_scale, cache.v_scale):
        t.copy_(torch.exp2(-torch.randint(6, 10, t.shape, generator=g, device="cuda").float()))


def shuffled_table(lens, page, n_pages, seed, spare=0):
    g = torch.Generator("cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    t = torch.full((len(lens), max(need + [1]) + spare), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = ids[at:at + k]
        at += k
    return t


def check_some(cache, got, q, table, lens, counts, which, scale, causal, window, layer=0):
    """The sequences `which` against the oracle, on copies of their pages."""
    d, page = q.shape[2], cache.k_codes.shape[3]
    first = np.concatenate([[0], np.cumsum(counts)])
    for b in which:
        n = -(-lens[b] // page)
        ids = table[b, :max(n, 1)].long().clamp(min=0)
        pool = P.Pool([codes_of(c[layer, ids]) for c in (cache.k_codes, cache.v_codes)],
                      [exps_of(s[layer, ids]) for s in (cache.k_scale, cache.v_scale)])
        rows = slice(int(first[b]), int(first[b + 1]))
        own = np.arange(max(n, 1), dtype=np.int32)[None]
        ref = P.attention(pool, q[rows].double().cpu().numpy(), own, [lens[b]], [counts[b]], scale, causal, window)
        check_attention([g[rows] for g in got], ref, d, lens[b], str((b, lens[b], counts[b])))


FORMS = [  # d, page, q heads, cache heads, lengths, query rows, window
    (128, 64, 4, 1, [9000], 1, 0),                                     # one item, the widest cluster
    (64, 16, 8, 2, [3000, 1, 0, 555], 2, 0),                           # clusters of eight
    (128, 32, 16, 8, [1200, 3, 900, 17, 1203], 1, 0),                  # clusters of two
    (64, 32, 16, 4, [700 - 20 * i for i in range(30)], 1, 0),          # one CTA an item
    (128, 128, 8, 8, [290] * 30, 1, 0),                                # two waves of them
    (128, 16, 16, 8, [(i * 37) % 601 for i in range(64)], 1, 0),       # equal runs of the line
    (128, 64, 32, 8, [(i * 131) % 1500 for i in range(50)], 4, 0),     # the same, two column tiles
    (64, 16, 24, 8, [4000 - 77 * i for i in range(50)], 1, 1000),      # the same, a window
    (128, 64, 8, 8, [0 if i % 7 == 3 else 5000 - 90 * i for i in range(50)], 1, 0),    # long runs
    (64, 128, 8, 4, [5000 - 90 * i for i in range(50)] + [1] * 300, 1, 0),             # more than 256 sequences
    (128, 32, 8, 1, [128 * (1 + i % 4) - i % 2 for i in range(160)], 5, 0),            # tensor cores, 1 to 4 tiles
    (64, 64, 8, 1, [1, 129, 2000, 257, 385], 9, 0),                    # the same, keys in ranges
    (64, 32, 16, 2, [1500, 90, 4000], 7, 300),                         # the same, a window
    (128, 16, 6, 2, [100, 700, 128, 1025], 60, 0),                     # two row tiles
]


@pytest.mark.parametrize("d,page,hq,hkv,lens,n,window", FORMS)
def test_attention_forms(d, page, hq, hkv, lens, n, window):
    n_pages = sum(-(-x // page) for x in lens) + 3
    cache = kvq.PagedCache.zeros(1, n_pages, hkv, page, d)
    fill(cache, d + len(lens))
    table = shuffled_table(lens, page, n_pages, 5, spare=2)
    counts = [n] * len(lens)
    g = torch.Generator("cuda").manual_seed(9)
    q = (torch.randn(n * len(lens), hq, d, generator=g, device="cuda") * 0.2).bfloat16()
    off = None if n == 1 else offsets_of(counts)
    got = kvq.paged_attention(cache, q, table, dev(lens), off, window=window, with_lse=True, max_q=n)
    clean()
    which = range(len(lens)) if len(lens) < 8 else sorted({0, 1, 3, len(lens) // 2, len(lens) - 2, len(lens) - 1})
    check_some(cache, got, q, table, lens, counts, which, 1 / np.sqrt(d), True, window)
    again = kvq.paged_attention(cache, q, table, dev(lens), off, window=window, with_lse=True, max_q=n)
    clean()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("d,hq,n,batch", [(128, 4, 1, 2), (64, 2, 7, 2), (128, 4, 1, 400), (64, 4, 10, 2),
                                          (128, 4, 90, 2), (128, 2, 150, 1)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_row_that_is_not_finite(d, hq, n, batch, bad):
    """A query row with a NaN or an infinity gives NaN; the others, those of
    its own head and tile among them, their results."""
    lens = [300 + b % 5 for b in range(batch)]
    n_pages = sum(-(-x // 64) for x in lens)
    cache = kvq.PagedCache.zeros(1, n_pages, 1, 64, d)
    fill(cache, 1)
    table = shuffled_table(lens, 64, n_pages, 2)
    counts = [n] * batch
    q = (torch.randn(n * batch, hq, d, generator=torch.Generator("cuda").manual_seed(8), device="cuda") * 0.3).bfloat16()
    at, head = n * batch // 2, hq - 1
    worse = q.clone()
    worse[at, head, 3] = bad
    clean_out = kvq.paged_attention(cache, q, table, dev(lens), offsets_of(counts), with_lse=True, max_q=n)
    got = kvq.paged_attention(cache, worse, table, dev(lens), offsets_of(counts), with_lse=True, max_q=n)
    clean()
    assert torch.isnan(got[0][at, head]).all() and torch.isnan(got[1][at, head])
    for g, c in zip(got, clean_out):
        g[at, head] = c[at, head]
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
    check_some(cache, got, q, table, lens, counts, [at // n], 1 / np.sqrt(d), True, 0)


@pytest.mark.parametrize("n,hq", [(8, 2), (40, 2)])
def test_widest_window(n, hq):
    """A window of 2^31 - 1 hides nothing, nor from rows before the first key."""
    cache = kvq.PagedCache.zeros(1, 4, 1, 16, 64)
    fill(cache, 6)
    lens = [2, 30]
    table = shuffled_table(lens, 16, 4, 7)
    q = torch.randn(2 * n, hq, 64, device="cuda").bfloat16()
    call = lambda w: kvq.paged_attention(cache, q, table, dev(lens), offsets_of([n, n]), max_q=n, causal=False, window=w,
                                         with_lse=True)
    a, b = call(0), call(0x7FFFFFFF)
    clean()
    assert torch.isfinite(a[1]).all() and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d,hq,n", [(128, 2, 30), (64, 4, 40), (128, 4, 60), (128, 8, 70)])
@pytest.mark.parametrize("step", [1, 40, 64, 100])
def test_scores_that_keep_growing(d, hq, n, step):
    """Keys whose scores climb by some binades every `step` keys, so that the
    softmax's base rises again and again, at any place of a tile."""
    page, length = 16, 1024
    cache = kvq.PagedCache.zeros(1, length // page, 1, page, d)
    fill(cache, 4)
    k = cache.k_codes.view(torch.uint8)
    k.zero_()
    grow = torch.arange(length, device="cuda") // step * step / 8.0       # 0 .. 128
    codes = (grow / 16).to(torch.float8_e4m3fn)                            # rounded as they are
    k[0, :, 0, :, 0] = codes.view(torch.uint8).view(length // page, page)
    cache.k_scale.fill_(1.0)
    q = (torch.randn(n, hq, d, generator=torch.Generator("cuda").manual_seed(3), device="cuda") * 0.1).bfloat16()
    q[:, :, 0] = 16.0
    table = torch.arange(length // page, dtype=torch.int32, device="cuda")[None]
    got = kvq.paged_attention(cache, q, table, dev([length]), offsets_of([n]), max_q=n, scale=1.0, with_lse=True)
    clean()
    check_some(cache, got, q, table, [length], [n], [0], 1.0, True, 0)


@pytest.mark.parametrize("n,hq", [(1, 4), (20, 2)])
def test_rows_behind_the_last_sequence_stay(n, hq):
    cache = kvq.PagedCache.zeros(1, 20, 2, 16, 64)
    fill(cache, 3)
    lens = [100, 60]
    table = shuffled_table(lens, 16, 20, 4)
    q = torch.randn(2 * n + 5, hq, 64, device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    off = dev([2, 2 + n, 2 + 2 * n])       # nor those before the first
    got = kvq.paged_attention(cache, q, table, dev(lens), off, max_q=n, out=out, with_lse=True)
    clean()
    assert (out[:2] == 7).all() and (out[2 + 2 * n:] == 7).all()
    rows = slice(2, 2 + 2 * n)
    check_some(cache, [g[rows] for g in got], q[rows], table, lens, [n, n], [0, 1], 0.125, True, 0)


def test_far_pages():
    """A pool of two layers, 5 GB of codes each for K and V: the same steps on
    pages at its end and on a small pool, bit for bit."""
    layers, heads, page, d, hq = 2, 8, 128, 128, 16
    n_far, n_near = 40000, 40
    far = kvq.PagedCache(*[torch.empty(layers, n_far, heads, page, d, dtype=torch.float8_e4m3fn, device="cuda")
                           for _ in range(2)],
                         *[torch.ones(layers, n_far, heads, dtype=torch.bfloat16, device="cuda") for _ in range(2)])
    near = kvq.PagedCache.zeros(layers, n_near, heads, page, d)
    ids = torch.arange(n_far - n_near, n_far, device="cuda").flip(0)   # near page i stands at ids[i]
    for t in (far.k_codes, far.v_codes):
        t.view(torch.uint8)[:, ids] = 0
    assert far.k_codes[0].numel() > 5 * 2 ** 30 - 2 ** 29
    lens = [700, 1290]
    near_t = torch.full((2, 13), -1, dtype=torch.int32, device="cuda")
    near_t[0, :6], near_t[1, :11] = torch.arange(6), torch.arange(6, 17)
    far_t = torch.where(near_t >= 0, ids[near_t.clamp(min=0).long()].to(torch.int32), near_t)
    g = torch.Generator("cuda").manual_seed(1)
    new = lambda rows, h: torch.randn(rows, h, d, generator=g, device="cuda").bfloat16()
    k, v, q1, q2 = new(sum(lens), heads), new(sum(lens), heads), new(2, hq), new(300, hq)
    k1, v1 = new(2, heads), new(2, heads)
    outs = []
    for cache, t in ((near, near_t), (far, far_t)):
        kvq.pages_append(cache, k, v, t, dev(lens), offsets_of(lens), layer=1)
        kvq.pages_append(cache, k1, v1, t, dev([x + 1 for x in lens]), layer=1)
        l = dev([x + 1 for x in lens])
        outs.append([*kvq.paged_attention(cache, q1, t, l, layer=1, with_lse=True),
                     *kvq.paged_attention(cache, q2, t, l, offsets_of([100, 200]), layer=1, max_q=200, with_lse=True)])
    clean()
    for a, b in zip(*outs):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    state = lambda c, at: [x[:, at].view(torch.uint8 if x.element_size() == 1 else torch.int16)
                           for x in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)]
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))
    assert same(state(near, torch.arange(17, device="cuda")), state(far, ids[:17]))
    # copies from the pool's end to its front and back
    last = int(ids[16])
    kvq.pages_copy(far, [last], [3])
    kvq.pages_copy(far, [3], [int(ids[30])])
    clean()
    one = lambda i: torch.tensor([i], device="cuda")
    assert same(state(far, one(last)), state(far, one(3))) and same(state(far, one(3)), state(far, one(int(ids[30]))))
    # all that lives moves to the front
    before = state(far, far_t[far_t >= 0].long())
    out, n_live = kvq.pages_compact(far, far_t)
    clean()
    assert int(n_live) == 17 and int(out.max()) == 16 and torch.equal(out < 0, far_t < 0)
    assert same(before, state(far, out[out >= 0].long()))


def test_two_graphs_replayed_together():
    """Two captured calls that take their workspaces from the binding, replayed
    on two streams at once: neither sees the other's."""
    lens = [[900 - i for i in range(64)], [1100 + i for i in range(64)]]
    sets = []
    for i, ln in enumerate(lens):
        n_pages = sum(-(-x // 64) for x in ln)
        cache = kvq.PagedCache.zeros(1, n_pages, 8, 64, 128)
        fill(cache, i)
        sets.append((cache, torch.randn(64, 16, 128, device="cuda").bfloat16(), shuffled_table(ln, 64, n_pages, i),
                     dev(ln)))
    assert sets[0][0].workspace_bytes(16, 64, sets[0][2].shape[1], 64, 1) > 16
    call = lambda s: kvq.paged_attention(*s, with_lse=True)
    want = [call(s) for s in sets]
    streams, graphs, got = [torch.cuda.Stream() for _ in sets], [], []
    torch.cuda.synchronize()
    for s, st in zip(sets, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            got.append(call(s))
        graphs.append(g)
    for _ in range(30):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    clean()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


CHILD = r'''
import torch
from quantized_kv_cache_quantize_gb300 import kvq
assert kvq.debug_bounds_build()
def clean(what):
    torch.cuda.synchronize()
    st, site = kvq.last_device_status(), kvq.debug_bounds_site()
    assert st == 0 and site == 0, (what, st, site)
for d, page, hq, hkv in ((128, 64, 8, 2), (64, 16, 3, 3)):
    for lens, n in (([300, 1, 65], 1), ([40] * 400, 1), ([90, 300], 9), ([260, 700], 140)):
        b = len(lens)
        width = -(-max(lens) // page)
        cache = kvq.PagedCache.zeros(2, b * width, hkv, page, d)
        table = torch.randperm(b * width, device="cuda").to(torch.int32).view(b, width)
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        new = lambda r, h: torch.randn(r, h, d, device="cuda").bfloat16()
        off = lambda c: torch.tensor([sum(c[:i]) for i in range(len(c) + 1)], dtype=torch.int32, device="cuda")
        kvq.pages_append(cache, new(sum(lens), hkv), new(sum(lens), hkv), table, ln, off(lens), layer=1)
        clean(("append", d, lens[0]))
        kvq.pages_append(cache, new(b, hkv), new(b, hkv), table, ln, layer=1)
        clean(("append one", d, lens[0]))
        c = [n] * b
        kvq.paged_attention(cache, new(n * b, hq), table, ln, off(c), layer=1, max_q=n, with_lse=True)
        clean(("attention", d, lens[0], n))
    kvq.pages_copy(cache, [0, 1], [5, 4])
    kvq.pages_compact(cache, table[:1])
    clean("pages")
print("checked build clean")
'''


def test_checked_build_runs_clean():
    from quantized_kv_cache_quantize_gb300 import build as b
    lib = b.build(checked=True)
    env = dict(os.environ, KVQ_LIBRARY=lib, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "checked build clean" in r.stdout
