"""The checked build runs rotations among views of one allocation, batches that
are mostly padding, and single rows next to masked keys without a failed check."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import torch
from quantized_kv_cache_quantize_gb300 import kvq
from tests import test_gpu_rope as R, test_gpu_rope_views as V, test_gpu_scored_masked as M, test_gpu_scored_padding as N

assert kvq.debug_bounds_build()

def clean(what):
    torch.cuda.synchronize()
    st, site = kvq.last_device_status(), kvq.debug_bounds_site()
    assert st == 0 and site == 0, (what, st, site)

for rows in (1, 9, 700):
    V.test_outputs_between_other_heads(rows)
V.test_outputs_between_other_heads_of_the_window()
for offsets in (False, True):
    V.test_append_writes_queries_beside_its_inputs(offsets)
for shape in R.SHAPES:
    R.test_packed(*shape, 301, 8, 3)
    R.test_packed(*shape, 1, 1, 1)
clean("rotations")
for case in N.PADDED:
    N.test_tiles_of_rows_that_see_nothing(*case, 5.0, 0.01)
    N.test_tiles_of_rows_that_see_nothing(*case, 5.0, 0.0)
N.test_nobody_sees_anything()
M.test_one_row_beside_masked_neighbours(128, 4, 20.0, 101, 130, 6.0, 0.01)
M.test_masked_places_decide_no_bit(128, 2, 200, 50.0, 0.0)
clean("scores")
print("checked build clean")
"""


def test_checked_build_runs_clean():
    from quantized_kv_cache_quantize_gb300 import build as b
    sources = glob.glob(os.path.join(b.CSRC, "*.cu*")) + glob.glob(os.path.join(b.CSRC, "*.h"))
    lib = b.CHECKED_LIB
    if not os.path.exists(lib) or os.path.getmtime(lib) < max(os.path.getmtime(s) for s in sources):
        b.build(checked=True)
    env = dict(os.environ, KVQ_LIBRARY=lib, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "checked build clean" in r.stdout
