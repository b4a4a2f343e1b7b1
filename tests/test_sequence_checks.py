"""Refusals of the linear-attention and layer-norm calls, on the CPU.

``sequence.cpp`` (argument checks, jobs, workspace sizes) is compiled as host
code together with stand-ins for the handle and the kernel launches, which
only count what would have been enqueued.  The driver calls the C ABI with
every kind of invalid argument and with layouts that must be taken."""
import os
import shutil
import subprocess

import pytest

from persistent_rnn_fwd_amd import build as buildmod

HERE = os.path.dirname(os.path.abspath(__file__))


def test_calls_refuse_what_they_cannot_run(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path / "sequence_checks")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-fsanitize=address,undefined",
           "-I" + os.path.join(buildmod.ROOT, "include"), "-I" + buildmod.CSRC, "-isystem", "/opt/rocm/include",
           os.path.join(HERE, "sequence_checks.cpp"), os.path.join(buildmod.CSRC, "sequence.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0, r.stdout + r.stderr[-3000:]
    assert "all checks passed" in r.stdout
