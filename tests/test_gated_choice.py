"""The gated feed-forward block's choice of kernels, on the CPU: the sizes that the GPU tests run
(_gated_tiles.py) reach every kernel that any size reaches, each with a reduction longer than its
ring, so that the ring's loop and the reuse of its slots run."""
import os
import random
import shutil
import subprocess

import pytest

from _gated_tiles import CASES, KERNELS, most

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = tmp_path_factory.mktemp("gated") / "gated_choice"
    subprocess.run(["g++", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-g", "-O1", "-std=c++17", "-Wall", "-I",
                    os.path.join(ROOT, "mixture_experts_layer_gemv_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "gated_choice.cpp"), "-o", str(exe)], check=True)

    def run(sizes, cus=256):
        """{kernel: stages of a share's reduction} of each (bf16, rows, m, p, experts)."""
        text = "\n".join(" ".join(map(str, map(int, (*s, cus)))) for s in sizes)
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr[-2000:]
        out = []
        for s, line in zip(sizes, r.stdout.splitlines(), strict=True):
            f, d = line.split(), {}
            for op, tile, splits, once, two, stages in zip(*(f[i::6] for i in range(6))):
                d[("bf16" if s[0] else "f32", op, tile, "once" if once == "1" else "kept", "split" if splits != "1" else "whole",
                   "two" if two == "1" else "one")] = int(stages), int(splits)
            out.append(d)
        return out

    return run


def test_the_sizes_cover_every_kernel_with_long_reductions(choice):
    covered = set()
    for (bf16, rows, m, p, E), kernels in zip(CASES.values(), choice(list(CASES.values()))):
        for kernel, (stages, splits) in kernels.items():
            if kernel[1] == "w":  # its reduction is an expert's rows: the fullest one's, of each part
                stages = -(-most(rows, E) // (64 if bf16 else 32)) * (2 if kernel[5] == "two" else 1)
            if stages // splits > int(kernel[2].rsplit("x", 1)[1]):
                covered.add(kernel)
    assert covered == KERNELS, KERNELS ^ covered


def test_no_size_takes_another_kernel(choice):
    """The whole range of the arguments, as far as the calls take them, under UndefinedBehaviorSanitizer."""
    g = random.Random(1)
    log = lambda lo, hi: int(lo * (hi / lo)**g.random())  # noqa: E731
    sizes = [(b, R, m, p, E) for b in (0, 1) for R in (1, 31, 33, 64, 2049, 1 << 20) for m in (8, 4096, 1 << 20)
             for p in (8, 14336, 1 << 20) for E in (1, 64)]
    sizes += [(g.randrange(2), log(1, 60000), 8 * log(1, 2048), 8 * log(1, 2048), g.choice((1, 2, 3, 5, 8, 16, 33, 64)))
              for _ in range(40000)]
    sizes = [s for s in sizes if (s[1] // 64 + s[4]) * -(-max(s[2:4]) // 128) < 1 << 22
             and 3 * s[4] * -(-s[2] // 128) * -(-s[3] // 128) < 1 << 23]
    seen = set().union(*choice(sizes))
    assert seen == KERNELS, seen ^ KERNELS
    for cus in (1, 104, 304):  # fewer or more CUs: no kernel that is not built
        assert {k[:3] for d in choice(sizes, cus) for k in d} <= {k[:3] for k in KERNELS}
