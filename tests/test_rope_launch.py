"""What the rotations' entry points work out on the host before a launch, checked
on the CPU (g++ on the library's own host headers)."""
import os
import shutil
import subprocess

import pytest

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
