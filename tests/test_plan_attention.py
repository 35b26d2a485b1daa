"""Host-only checks of the plans and workspace layouts of the attention,
rotary and 4-bit cache entry points
(integer_only_dnn_amd/csrc/ie_plan.cpp), compiled with g++ under the address
and undefined-behaviour sanitizers together with tests/plan_attention_check.cpp.
No GPU is involved."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = [os.path.join(ROOT, "tests", "plan_attention_check.cpp"),
       os.path.join(ROOT, "integer_only_dnn_amd", "csrc", "ie_plan.cpp")]


def test_attention_plans_and_workspace_layouts_under_sanitizers(tmp_path):
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "plan_attention_check")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", *SRC, "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-4000:]
    env = {k: v for k, v in os.environ.items() if k not in ("IE_TILE", "IE_WTILE")}
    env.update(ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert res.returncode == 0, (res.stdout + res.stderr)[-4000:]
    assert "plan_attention_check:" in res.stdout
