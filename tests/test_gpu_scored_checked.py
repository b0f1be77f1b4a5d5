"""The checked build (every kernel tests its indices) runs rotary positions, the
append that rotates and attention with shaped scores without a failed check, in a
child process that loads it through KVQ_LIBRARY; the results are the oracle's."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import numpy as np, torch
from quantized_kv_cache_quantize_gb300 import kvq
from tests import test_gpu_rope as R, test_gpu_scored as S

assert kvq.debug_bounds_build()

def clean(what):
    torch.cuda.synchronize()
    st, site = kvq.last_device_status(), kvq.debug_bounds_site()
    assert st == 0 and site == 0, (what, st, site)

for case in S.CASES:
    S.run_case(*case)
    clean(case)
S.test_what_no_row_sees_does_not_matter(128, 128, 2, 70, 8.0)
S.test_many_short_sequences(64, 6, 3, 2, 5.0, True, True, 4)
for case in R.APPENDS:
    R.test_append(*case, True)
    clean(case)
R.test_packed(128, 64, [22, 21, 21], True, 301, 8, 3)
R.test_window_layout(64, 32, [8, 8, 8, 8], False, False)
R.test_rows_outside_the_offsets_are_left(True)
clean("rope")
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
