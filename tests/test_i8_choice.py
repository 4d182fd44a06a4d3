"""The int8 product's choice of a kernel, on the CPU: the GPU tests' sizes for
each kernel do select it, and they cover all of them."""
import os
import shutil
import subprocess

import pytest

from _i8_tiles import CASES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KERNELS = ["32x256x3", "64x256x3", "32x256x2", "64x256x2", "256x256x2", "128x256x3", "128x128x4", "64x128x3", "64x64x4",
           "ring16", "ring64", "ring32"]


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = tmp_path_factory.mktemp("i8") / "i8_choice"
    subprocess.run(["g++", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-g", "-O1", "-std=c++17", "-Wall", "-I",
                    os.path.join(ROOT, "mixture_experts_layer_gemv_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "i8_choice.cpp"), "-o", str(exe)], check=True)

    def run(sizes, cus=256):
        text = "\n".join(" ".join(map(str, (*s, cus))) for s in sizes)
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr[-2000:]
        out = [l.split() for l in r.stdout.splitlines()]
        assert len(out) == len(sizes)
        return [(k, a == "1", b == "1") for k, a, b in out]

    return run


def test_each_size_selects_its_kernel(choice):
    got = choice([(sum(c), K, N, len(c)) for c, K, N, *_ in CASES.values()])
    want = [tuple(v[3:]) for v in CASES.values()]
    assert got == want, {n: (g, w) for n, g, w in zip(CASES, got, want) if g != w}


def test_the_sizes_cover_every_kernel():
    assert {(v[3], v[5]) for v in CASES.values()} == {(k, b) for k in KERNELS for b in (False, True)}
    for k in ("256x256x2", "128x256x3", "128x128x4", "64x128x3", "64x64x4"):  # the others only ever read weights once
        assert {v[4] for v in CASES.values() if v[3] == k} == {False, True}
    for name, (counts, K, N, kernel, *_) in CASES.items():
        stages, ring = -(-K // 128), 2 if kernel.startswith("ring") else int(kernel.rsplit("x", 1)[1])
        waves = 4 if kernel.startswith("ring") else 1  # a ring's wave takes a quarter of the stages
        assert stages // waves > ring, name


def test_every_size_has_a_kernel(choice):
    """The whole range of rows, channels, experts (as far as the call takes them) and CUs, under UndefinedBehaviorSanitizer."""
    sizes = [(R, K, N, E) for R in (1, 2, 15, 16, 17, 63, 64, 65, 777, 16384, 1 << 24, 1 << 30) for K in (16, 4096, 131056)
             for N in (8, 136, 4096, 1 << 20, 2**28 - 16) for E in (1, 2, 63, 64) if (R // 64 + E) * -(-N // 16) < 1 << 24]
    for cus in (1, 104, 256, 304):
        assert {k for k, _, _ in choice(sizes, cus)} <= set(KERNELS)
