"""Builds and runs tests/native/gated_banks_check.cpp: the LDS banks of the gated feed-forward
block's fp32 reads (those of its transposing reads are in gated_index_check.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_gated_banks(tmp_path):
    exe = tmp_path / "gated_banks_check"
    subprocess.run(["g++", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g", "-O1", "-std=c++17", "-Wall",
                    "-I", os.path.join(ROOT, "mixture_experts_layer_gemv_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "gated_banks_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "gated banks check ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
