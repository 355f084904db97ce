"""After an error the next call finds the join counters cleared (tests/c/kv_recovery.cpp, on the host)."""
import os
import subprocess

from indexer_topk_long_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_counters_are_cleared_after_any_error(ltk_lib, tmp_path):
    exe = str(tmp_path / "kv_recovery")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    build = subprocess.run(
        ["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), "-I", cuda, os.path.join(ROOT, "tests", "c", "kv_recovery.cpp"),
         os.path.join(_build.BUILD, "kv_api.o"), "-o", exe], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and run.stdout.strip() == "recovery ok", run.stdout + run.stderr
