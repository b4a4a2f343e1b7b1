"""Refusals and plans of the gated delta rule and rms norm, on the CPU.

Their host sources (argument checks, segments, workspace) are compiled as host
code together with stand-ins for the handle and the kernel launches, which keep
what would have been enqueued."""
import os
import shutil
import subprocess

import pytest

from persistent_rnn_fwd_amd import build as buildmod

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path_factory.mktemp("delta") / "delta_checks")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-fsanitize=address,undefined",
           "-I" + os.path.join(buildmod.ROOT, "include"), "-I" + buildmod.CSRC, "-isystem", "/opt/rocm/include",
           os.path.join(HERE, "delta_checks.cpp"), *(os.path.join(buildmod.CSRC, s) for s in ("delta_calls.cpp", "rms_calls.cpp")),
           "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


@pytest.mark.parametrize("what", ["delta refusals", "delta plans", "rms refusals"])
def test_calls(driver, what):
    r = subprocess.run([driver, what], capture_output=True, text=True, env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "all checks passed" in r.stdout
