"""Host-only checks of the block operators' launches: integer_only_dnn_amd/csrc/ie_plan.cpp
compiled with g++ together with tests/plan_launch_check.cpp."""

import ctypes
import os
import shutil
import subprocess

import pytest

from integer_only_dnn_amd import ie
from tests import test_gpu_trips

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = [os.path.join(ROOT, "tests", "plan_launch_check.cpp"),
       os.path.join(ROOT, "integer_only_dnn_amd", "csrc", "ie_plan.cpp")]


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    """Runs the check with the arguments given; it has to pass."""
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("plan") / "plan_launch_check")
    res = subprocess.run([cxx, "-std=c++17", "-O1", *SRC, "-o", exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-4000:]
    env = {k: v for k, v in os.environ.items() if k not in ("IE_TILE", "IE_WTILE")}

    def run(*args):
        res = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=300, env=env)
        assert res.returncode == 0, (res.stdout + res.stderr)[-4000:]
        assert "plan_launch_check:" in res.stdout
    return run


def test_block_launches(check):
    check()


@pytest.mark.parametrize("kind,shapes", [("forward", test_gpu_trips.NORM), ("backward", test_gpu_trips.NORM),
                                         ("dropout", test_gpu_trips.DROPOUT)], ids=["forward", "backward", "dropout"])
def test_gpu_shapes_take_every_split_to_a_second_trip(check, kind, shapes):
    check(kind, *[n for s in shapes for n in s])


@pytest.mark.parametrize("name,args", [("launch_norm_fwd", "7NormFwd"), ("launch_norm_bwd", "7NormBwd"),
                                       ("launch_dropout", "8DropArgs")])
def test_a_split_without_a_kernel_is_an_error(name, args):
    """Nothing launched is not success: hipErrorInvalidValue (1), before any call of the runtime."""
    launch = getattr(ie.lib(), f"_ZN2ie{len(name)}{name}ERKNS_{args}ERKNS_8NormPlanEP12ihipStream_t")
    plan = (ctypes.c_int * 3)(7, 4, 1)
    for mode in range(4):
        block = (ctypes.c_int * 256)(*[mode] * 256)  # the mode wherever it lies
        assert launch(block, plan, None) == 1
