"""What linear attention launches, on the CPU: the host side (``sequence.cpp``,
``attention_plan.cpp``) with stand-ins for the handle and the launches, which
keep the arguments for the driver to check."""
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
    exe = str(tmp_path_factory.mktemp("jobs") / "attention_jobs")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-I" + os.path.join(buildmod.ROOT, "include"), "-I" + buildmod.CSRC, "-isystem", "/opt/rocm/include",
           os.path.join(HERE, "attention_jobs.cpp"), os.path.join(buildmod.CSRC, "sequence.cpp"),
           os.path.join(buildmod.CSRC, "attention_plan.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


@pytest.mark.parametrize("what", ["long sequences", "gradients in place", "shared heads", "packed workspace", "wide norms", "grids", "spans"])
def test_launches(driver, what):
    r = subprocess.run([driver, what], capture_output=True, text=True, env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "all checks passed" in r.stdout
