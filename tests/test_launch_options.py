"""Launch options (shared memory above 48 KB, wide clusters): asked for once per kernel and
device, right with several threads (no GPU: the runtime is a stand-in)."""
import os
import subprocess

import pytest

from moe_expert_ffn_top_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("native") / "launch_options")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build._nvcc()))), "include")
    cmd = ["g++", "-std=c++17", "-pthread", "-I", cuda, "-o", exe, os.path.join(HERE, "native", "launch_options.cpp"),
           "-x", "c++", os.path.join(_build.CSRC, "options.cu")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("what", ["race", "no_lowering", "devices", "again"])
def test_launch_options(program, what):
    r = subprocess.run([program, what], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
