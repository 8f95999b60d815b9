"""The planner's arithmetic with KV tiles from spans of each query, compiled for the host: every item and partial row has room."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_kv_cache_168_gb300", "csrc")


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_every_item_and_partial_row_has_room(tmp_path, seed):
    exe = str(tmp_path / "extend_spans_check")
    subprocess.run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, os.path.join(HERE, "extend_spans_check.cpp"), "-o", exe],
                   check=True)
    r = subprocess.run([exe, str(seed), "4000"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-4000:]
