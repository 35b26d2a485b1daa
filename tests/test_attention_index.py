"""Which workgroup of attention takes which tile and head: the kernels' own index arithmetic, compiled for the host with the
lanes of a wave written out (tests/attention_index_check.cpp); up to 10000 sequences under the address and
undefined-behaviour sanitizers, up to 300000 without them."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "attention_index_check.cpp")


@pytest.mark.parametrize("flags,args", [(["-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all"], []), (["-O2"], ["large"])],
                         ids=["sanitized", "large"])
def test_every_tile_is_met_once(tmp_path, flags, args):
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "attention_index_check")
    res = subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", *flags, SRC, "-o", exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-4000:]
    res = subprocess.run([exe, *args], capture_output=True, text=True, timeout=300, env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert res.returncode == 0, (res.stdout + res.stderr)[-4000:]
    assert "attention_index_check:" in res.stdout
