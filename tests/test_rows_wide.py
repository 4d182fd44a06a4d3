"""Builds and runs tests/native/rows_wide_check.cpp: the columns of the row
operators for rows up to the widest that an int counts, checked on the CPU
under UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_columns_of_wide_rows(tmp_path):
    exe = tmp_path / "rows_wide_check"
    subprocess.run(["g++", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-g", "-O1", "-std=c++17", "-Wall", "-I",
                    os.path.join(ROOT, "mixture_experts_layer_gemv_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "rows_wide_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "wide rows ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
