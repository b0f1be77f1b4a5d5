"""The scratch that the paged calls take when they are given none: held until
the library has launched all its kernels, and a call's own where two host
threads name the same stream."""
from __future__ import annotations

import threading
import weakref

import pytest
import torch

from quantized_kv_cache_quantize_gb300 import kvq

pytestmark = pytest.mark.gpu


def line_case(seed, batch=64, length=900):
    """A decoding step that goes through the workspace, in two kernels."""
    n = -(-length // 64)
    cache = kvq.PagedCache.zeros(1, batch * n, 8, 64, 128)
    g = torch.Generator("cuda").manual_seed(seed)
    for t in (cache.k_codes, cache.v_codes):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(torch.float8_e4m3fn))
    table = torch.randperm(batch * n, generator=g, device="cuda").to(torch.int32).view(batch, n)
    lens = torch.randint(1, length + 1, (batch,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(batch, 16, 128, generator=g, device="cuda").bfloat16()
    assert cache.workspace_bytes(16, batch, n, batch, 1) > 16
    return cache, lambda **kw: kvq.paged_attention(cache, q, table, lens, with_lse=True, **kw)


def split_case(seed):
    """Many rows of one sequence, its keys in ranges that a second kernel joins."""
    cache = kvq.PagedCache.zeros(1, 64, 2, 64, 128)
    g = torch.Generator("cuda").manual_seed(seed)
    for t in (cache.k_codes, cache.v_codes):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(torch.float8_e4m3fn))
    table = torch.randperm(64, generator=g, device="cuda").to(torch.int32).view(1, 64)
    lens = torch.tensor([4090], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    q = torch.randn(40, 4, 128, generator=g, device="cuda").bfloat16()
    assert cache.workspace_bytes(4, 1, 64, 40, 40) > 16
    return cache, lambda **kw: kvq.paged_attention(cache, q, table, lens, off, max_q=40, with_lse=True, **kw)


def compact_case(seed):
    cache = kvq.PagedCache.zeros(2, 300, 1, 16, 64)
    g = torch.Generator("cuda").manual_seed(seed)
    cache.k_codes.copy_(torch.randn(cache.k_codes.shape, generator=g, device="cuda").to(torch.float8_e4m3fn))
    table = torch.randperm(300, generator=g, device="cuda").to(torch.int32)[:150].view(5, 30).contiguous()
    return cache, lambda **kw: kvq.pages_compact(cache, table, **kw)


class Watched:
    """The library, with a look at the scratch before the calls that take it."""

    def __init__(self, real, look):
        self.real, self.look = real, look

    def __getattr__(self, name):
        f = getattr(self.real, name)
        if name not in ("kvq_paged_attention", "kvq_pages_compact"):
            return f

        def call(*args):
            self.look()
            return f(*args)
        return call


@pytest.mark.parametrize("case", [line_case, split_case, compact_case])
@pytest.mark.parametrize("how", ["named stream", "captured", "kept scratch let go by another thread"])
def test_scratch_is_held_until_the_call_returns(case, how, monkeypatch):
    cache, call = case(1)
    call()
    torch.cuda.synchronize()
    taken, seen = [], []
    make = kvq.PagedCache._workspace

    def workspace(self, *args):
        t = make(self, *args)
        taken.append(weakref.ref(t))
        return t

    def look():
        if how.startswith("kept"):
            cache._workspaces.clear()
        seen.append(taken[-1]() is not None)
    monkeypatch.setattr(kvq.PagedCache, "_workspace", workspace)
    watched = Watched(kvq.lib(), look)
    monkeypatch.setattr(kvq, "lib", lambda: watched)
    stream = torch.cuda.Stream()
    if how == "captured":
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=stream):
            call()
    else:
        call(**(dict(stream=stream) if how == "named stream" else {}))
    torch.cuda.synchronize()
    assert seen == [True]


@pytest.mark.parametrize("case,rounds", [(line_case, 60), (split_case, 60), (compact_case, 1)])
def test_two_host_threads_on_one_named_stream(case, rounds):
    """Both threads' calls on the same stream, each with scratch of its own:
    the results of the calls one after another, bit for bit."""
    sets = [case(2), case(3)]
    want = [call() for _, call in (case(2), case(3))]
    torch.cuda.synchronize()
    stream, got, start = torch.cuda.Stream(), [[], []], threading.Barrier(2)

    def work(i):
        start.wait()
        for _ in range(rounds):
            got[i].append(sets[i][1](stream=stream))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert kvq.last_device_status() == kvq.KVQ_OK
    for i in range(2):
        assert len(got[i]) == rounds
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
