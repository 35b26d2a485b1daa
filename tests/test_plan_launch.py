"""Host-only checks of the block operators' launches: integer_only_dnn_amd/csrc/ie_plan.cpp
compiled with g++ together with tests/plan_launch_check.cpp."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = [os.path.join(ROOT, "tests", "plan_launch_check.cpp"),
       os.path.join(ROOT, "integer_only_dnn_amd", "csrc", "ie_plan.cpp")]


def test_block_launches(tmp_path):
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "plan_launch_check")
    res = subprocess.run([cxx, "-std=c++17", "-O1", *SRC, "-o", exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-4000:]
    env = {k: v for k, v in os.environ.items() if k not in ("IE_TILE", "IE_WTILE")}
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert res.returncode == 0, (res.stdout + res.stderr)[-4000:]
    assert "plan_launch_check:" in res.stdout
