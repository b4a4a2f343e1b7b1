"""Grids of the gated delta rule's launches, on the CPU (see delta_grid_checks.cpp)."""
import os
import shutil
import subprocess

import pytest

from persistent_rnn_fwd_amd import build as buildmod

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_launch_counts_its_threads_in_32_bits(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path / "delta_grid_checks")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-Wno-unused-function", "-D__HIP_PLATFORM_AMD__",
           "-fsanitize=address,undefined", "-I" + os.path.join(buildmod.ROOT, "include"), "-I" + buildmod.CSRC, "-I" + HERE,
           "-isystem", "/opt/rocm/include", os.path.join(HERE, "delta_grid_checks.cpp"),
           *(os.path.join(buildmod.CSRC, s) for s in ("delta_calls.cpp", "rms_calls.cpp")), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "all checks passed" in r.stdout
