"""The arithmetic by which pa_extend's planner cuts a call into items (csrc/extend_plan.h), compiled for the host: every
item and partial row has room in the workspace, and a query tile's parts cover its KV tiles exactly once."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_kv_cache_168_gb300", "csrc")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "extend_plan_check")
    cxx = shutil.which("g++") or "g++"
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, os.path.join(HERE, "extend_plan_check.cpp"), "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("heads", [0, 1, 2])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_every_item_and_partial_row_has_room(program, seed, heads):
    r = subprocess.run([program, str(seed), "3000", str(heads)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-4000:]
