"""Host-side book of the expert products' tile counters (tests/c/tile_counters.cpp)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "combine_get_dispatch_02_gb300", "csrc")


def test_counters_are_exclusive_and_come_back(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path / "tile_counters")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
           os.path.join(HERE, "c", "tile_counters.cpp"), "-o", exe, "-pthread"]
    if subprocess.run(cmd + ["-fsanitize=address"], capture_output=True).returncode != 0:
        subprocess.run(cmd, check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
