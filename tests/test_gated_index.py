"""Builds and runs tests/native/gated_index_check.cpp: the index arithmetic of
the gated feed-forward block, checked exhaustively on the CPU under
AddressSanitizer and UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_gated_index_math(tmp_path):
    exe = tmp_path / "gated_index_check"
    subprocess.run(["g++", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g", "-O1", "-std=c++17", "-Wall",
                    "-I", os.path.join(ROOT, "mixture_experts_layer_gemv_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "gated_index_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "gated index check ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
