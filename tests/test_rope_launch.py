"""What the rotations' entry points work out on the host before a launch, checked
on the CPU (g++ on the library's own host headers)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from quantized_kv_cache_quantize_gb300 import kvq
from tests.test_paged_host import PTR, _pages, _seqs

HERE = os.path.dirname(os.path.abspath(__file__))


def run(tmp_path, source):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = os.path.join(tmp_path, "check")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-I", cuda, "-o", exe, os.path.join(HERE, source)])
    out = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "bad 0" in out.stdout, out.stdout + out.stderr


def test_blocks_of_any_size(tmp_path):
    run(tmp_path, "rope_blocks_check.cpp")


def test_overlap_of_strided_tensors(tmp_path):
    run(tmp_path, "overlap_check.cpp")


# ---- the entry points refuse what overlaps ----

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kvq.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return kvq.lib()


def _tensor(x, y, heads, row=6144, head=128):
    return kvq.RopeTensorStruct(PTR + 2 * x, PTR + 2 * y, 0, row, head, 0, row, head, heads)


@pytest.mark.parametrize("q,k", [
    ((0, 8 * 128, 32), (32 * 128, 1 << 30, 8)),                  # queries' output over their own inputs
    ((0, 1 << 30, 32), (32 * 128, 8 * 128, 8)),                  # keys' output over the queries
    ((0, 16 * 128, 8), (20 * 128, 1 << 30, 8)),                  # queries' output over half the keys
    ((0, 1 << 30, 8), (8 * 128, (1 << 30) + 7 * 128, 8)),        # outputs over one another
    ((0, 6144, 8), (8 * 128, 1 << 30, 8)),                       # a row further on
    ((0, 6144 * 9, 8), (8 * 128, 1 << 30, 8)),                   # over the last row
])
def test_rotation_refuses_overlaps(lib, q, k):
    t = kvq.RopeTableStruct()
    t.cos_sin, t.n_positions, t.pairs, t.axes = PTR + (1 << 40), 100, 32, 1
    a = (kvq.RopeTensorStruct * 2)(_tensor(*q), _tensor(*k))
    assert lib.kvq_rope(ctypes.byref(t), PTR + (1 << 40), 0, 1, 0, 1, 10, 128, 0, a, 2, None) == kvq.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("shift", [128, 7 * 128, 6144, 9 * 6144, 9 * 6144 + 7 * 128])
def test_rotation_refuses_a_shifted_place(lib, shift):
    """An output neither in place nor apart: some heads or rows further on."""
    t = kvq.RopeTableStruct()
    t.cos_sin, t.n_positions, t.pairs, t.axes = PTR + (1 << 40), 100, 32, 1
    for x, y in ((0, shift), (shift, 0)):
        a = _tensor(x, y, 8)
        assert lib.kvq_rope(ctypes.byref(t), PTR + (1 << 40), 0, 1, 0, 1, 10, 128, 0, ctypes.byref(a), 1, None) == kvq.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("row,head", [(0, 128), (1016, 128), (6144, 0), (6144, 64)])
def test_outputs_that_repeat_memory(lib, row, head):
    """Rows or heads of an output on top of one another, in place or not."""
    t = kvq.RopeTableStruct()
    t.cos_sin, t.n_positions, t.pairs, t.axes = PTR + (1 << 40), 100, 32, 1
    for x in (1 << 30, 0):
        a = _tensor(x, 1 << 30, 8, row, head)
        assert lib.kvq_rope(ctypes.byref(t), PTR + (1 << 40), 0, 1, 0, 1, 10, 128, 0, ctypes.byref(a), 1, None) == kvq.KVQ_ERR_INVALID_ARG
    args = [ctypes.byref(_pages()), 0, ctypes.byref(t), None, 0, PTR, 512, 128, PTR, 512, 128,
            PTR + (1 << 31), 6144, 128, 8, PTR + (1 << 32), row, head, ctypes.byref(_seqs()), None]
    assert lib.kvq_pages_append_rope(*args) == kvq.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("out", [128, 31 * 128, 32 * 128 + 7 * 128, 40 * 128 + 3 * 128, 6144 * 2, 6144 + 47 * 128])
def test_append_refuses_overlaps(lib, out):
    """One projection of 48 heads a row: 32 of queries, 8 of keys, 8 of values."""
    t = kvq.RopeTableStruct()
    t.cos_sin, t.n_positions, t.pairs, t.axes = PTR + (1 << 40), 100, 32, 1
    args = [ctypes.byref(_pages()), 0, ctypes.byref(t), None, 0, PTR + 2 * 32 * 128, 6144, 128, PTR + 2 * 40 * 128, 6144, 128,
            PTR, 6144, 128, 32, PTR + 2 * out, 6144, 128, ctypes.byref(_seqs()), None]
    assert lib.kvq_pages_append_rope(*args) == kvq.KVQ_ERR_INVALID_ARG
