"""moe_matmul_i8 and moe_quantize_codes_i8 against the definition in 64 bits.

The int32 sum is exact, so an output differs from the exact value by the
roundings of its conversion to fp32 (u = 2^-24 relative), of the two scale
products (u each) and of the store (half a step of the output type).
"""
import numpy as np
import pytest
import torch

import oracle
import mixture_experts_layer_gemv_amd as M

from _gpu import log

pytestmark = pytest.mark.gpu

u = 2.0**-24
U = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8}
CODE = {torch.float32: M.MOE_F32, torch.bfloat16: M.MOE_BF16}
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


def codes(shape, seed, lo=-127, hi=127):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=g, dtype=torch.int8, device="cuda")


def scales(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(shape, generator=g, device="cuda") + 0.5) * 0.01


def exact(x, sx, w, sw, offsets, perm, topk, rows):
    """y in 64 bits; NaN where no expert has the row."""
    E, N, _ = w.shape
    y = torch.full((rows, N), float("nan"), dtype=torch.float64, device="cuda")
    for e in range(E):
        lo, hi = (0, rows) if offsets is None else (int(offsets[e]), int(offsets[e + 1]))
        at = torch.arange(lo, hi, device="cuda")
        t = at if perm is None else perm.long()[at] // topk
        if hi > lo:
            y[lo:hi] = (x[t].double() @ w[e].double().t()) * sx[t].double()[:, None] * sw[e].double()
    return y


def run(x, sx, w, sw, offsets, perm, topk, rows, out):
    E, N, K = w.shape
    buf = torch.full((rows * N + 128,), 7.0, dtype=out, device="cuda")
    y = buf[64:64 + rows * N].view(rows, N)
    M.moe_matmul_i8(x, sx, w, sw, offsets, perm, len(x), topk, rows, K, N, E, y, CODE[out])
    torch.cuda.synchronize()
    assert bool((buf[:64] == 7).all()) and bool((buf[64 + rows * N:] == 7).all())
    return y


def check(y, ref, out, what=""):
    rows = ~torch.isnan(ref).any(1)
    assert bool((y[~rows] == 7).all()), "rows of no expert were written"
    err, r = (y[rows].double() - ref[rows]).abs(), ref[rows].abs()
    bar = r * (U[out] + 3 * u) * (1 + 2.0**-7) + 1e-37
    log(f"  {what}: {float((err / bar).max()) if err.numel() else 0:.3f} of the bound")
    assert bool((err <= bar).all()), what


DENSE = [(1, 16, 8), (1, 64, 16), (3, 48, 24), (16, 4096, 512), (17, 80, 40), (64, 256, 1000), (65, 1040, 264),
         (100, 16, 4104), (128, 512, 256), (200, 2048, 520), (257, 272, 776), (511, 1024, 1032), (1003, 656, 2048),
         (1500, 144, 4096), (2049, 4096, 1000), (4100, 528, 1288)]


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,K,N", DENSE)
def test_dense(R, K, N, out):
    log(f"matmul_i8 dense R={R} K={K} N={N} {out}")
    x, w, sx, sw = codes((R, K), R + K), codes((1, N, K), N), scales((R,), 1), scales((1, N), 2)
    check(run(x, sx, w, sw, None, None, 1, R, out), exact(x, sx, w, sw, None, None, 1, R), out, "y")


# wide enough for every tile shape the launch chooses from on 256 CUs: 256 x
# 256, 128 x 256, 128 x 128, 64 x 128, 64 x 64 and 32 x 256 rows by channels, and the two
# kernels for few rows; K with and without a partial last stage
WIDE = [(4100, 144, 4104), (3841, 384, 4360), (2049, 272, 4104), (2300, 256, 3080), (515, 208, 4008), (450, 640, 4104),
        (300, 400, 8200), (1030, 272, 3080), (60, 176, 12296), (64, 256, 12808), (31, 400, 2056), (32, 2064, 136), (16, 4112, 1032), (40, 2064, 72)]


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,K,N", WIDE)
def test_dense_tiles(R, K, N, out):
    log(f"matmul_i8 dense R={R} K={K} N={N} {out}")
    x, w, sx, sw = codes((R, K), R + K), codes((1, N, K), N), scales((R,), 1), scales((1, N), 2)
    check(run(x, sx, w, sw, None, None, 1, R, out), exact(x, sx, w, sw, None, None, 1, R), out, "y")


def grouped(counts, k, seed):
    """offsets and a perm of a token set of ceil(rows / k) tokens."""
    g = torch.Generator().manual_seed(seed)
    rows = sum(counts)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), device="cuda")
    T = (rows + k - 1) // k
    perm = torch.randperm(T * k, generator=g)[:rows].to(torch.int32).cuda()
    return offsets, perm, T, rows


COUNTS = {"one_row": [0, 1, 0], "empty_ends": [0, 5, 0, 17, 0], "decode": [4, 1, 0, 7, 2, 16, 9, 1],
          "hot": [200, 1, 0, 3], "mixed": [64, 65, 63, 128, 1, 0, 15, 16], "large": [300, 257, 1, 512, 700, 0, 255, 31],
          "e64": [i % 5 for i in range(64)], "even": [256, 256]}


@pytest.mark.parametrize("gather", [True, False], ids=["gather", "sorted"])
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("K,N", [(64, 128), (528, 200), (2048, 768)])
@pytest.mark.parametrize("counts", COUNTS)
def test_experts(counts, K, N, out, gather):
    c = COUNTS[counts]
    k = 2
    offsets, perm, T, rows = grouped(c, k, len(c))
    log(f"matmul_i8 experts {counts} K={K} N={N} {out} gather={gather}")
    if not gather:
        perm, T = None, rows
    x, w, sx, sw = codes((T, K), K), codes((len(c), N, K), N), scales((T,), 1), scales((len(c), N), 2)
    check(run(x, sx, w, sw, offsets, perm, k, rows, out), exact(x, sx, w, sw, offsets, perm, k, rows), out, "y")


# (counts, K, N): the same for experts
WIDE_EXPERTS = {"256x256": ([300, 257, 1, 512, 700, 0, 255, 31], 272, 3208), "128x256": ([64, 200, 129, 0, 1, 128, 127, 99], 400, 6280),
                "64x128": ([40, 65, 64, 0, 33, 90, 1, 47], 256, 3336), "32x256": ([4, 33, 0, 17, 32, 1, 16, 90], 384, 12296),
                "32x256_tail": ([4, 1, 0, 17, 32, 1, 16, 3], 144, 12808), "64x64": ([4, 33, 0, 17, 32, 1, 16, 90], 528, 2056),
                "16": ([3, 1, 0, 17, 16, 1, 5, 2], 2064, 200), "32": ([64, 1, 0, 33, 80], 2064, 200)}


@pytest.mark.parametrize("gather", [True, False], ids=["gather", "sorted"])
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", WIDE_EXPERTS)
def test_experts_tiles(name, out, gather):
    c, K, N = WIDE_EXPERTS[name]
    offsets, perm, T, rows = grouped(c, 2, len(c))
    log(f"matmul_i8 experts {name} {out} gather={gather}")
    if not gather:
        perm, T = None, rows
    x, w, sx, sw = codes((T, K), K), codes((len(c), N, K), N), scales((T,), 1), scales((len(c), N), 2)
    check(run(x, sx, w, sw, offsets, perm, 2, rows, out), exact(x, sx, w, sw, offsets, perm, 2, rows), out, "y")


@pytest.mark.parametrize("R,N", [(5, 64), (300, 520)])
def test_extreme_sums(R, N):
    """Codes of -128 and 127 at the longest K: the largest sums int32 has to hold."""
    K = 131056
    x, w = torch.full((R, K), -128, dtype=torch.int8, device="cuda"), torch.full((1, N, K), -128, dtype=torch.int8,
                                                                               device="cuda")
    w[:, 1::2] = 127
    sx, sw = torch.ones(R, device="cuda"), torch.ones(1, N, device="cuda")
    y = run(x, sx, w, sw, None, None, 1, R, F32)
    even, odd = 128.0 * 128 * K, -128.0 * 127 * K
    assert bool((y[:, 0::2].double() - even).abs().max() <= u * even)
    assert bool((y[:, 1::2].double() - odd).abs().max() <= u * -odd)


@pytest.mark.parametrize("R", [6, 400])
def test_rows_of_no_range_and_clamped_inputs(R):
    """Rows before the first range, between and behind the ranges stay as they
    were; offsets and permutation entries outside their range are clamped."""
    K, N, E = 128, 64, 3
    x, w, sx, sw = codes((R, K), 1), codes((E, N, K), 2), scales((R,), 3), scales((E, N), 4)
    offsets = torch.tensor([1, 3, 3, R - 2], dtype=torch.int32, device="cuda")
    check(run(x, sx, w, sw, offsets, None, 1, R, F32), exact(x, sx, w, sw, offsets, None, 1, R), F32)
    wild = torch.tensor([-5, 3, 2**31 - 1, R + 7], dtype=torch.int32, device="cuda")  # [0,3) [3,R) [R,R)
    tame = torch.tensor([0, 3, R, R], dtype=torch.int32, device="cuda")
    check(run(x, sx, w, sw, wild, None, 1, R, F32), exact(x, sx, w, sw, tame, None, 1, R), F32)
    falling = torch.tensor([2, 5, 3, R], dtype=torch.int32, device="cuda")  # [2,5) [5,5) [5,R)
    tame = torch.tensor([2, 5, 5, R], dtype=torch.int32, device="cuda")
    check(run(x, sx, w, sw, falling, None, 1, R, F32), exact(x, sx, w, sw, tame, None, 1, R), F32)
    tame = torch.tensor([0, 3, R, R], dtype=torch.int32, device="cuda")
    perm = torch.arange(R, dtype=torch.int32, device="cuda")
    perm[0], perm[1], perm[R - 1] = -7, R + 100, 2**31 - 1
    tame_p = perm.clamp(0, R - 1)
    check(run(x, sx, w, sw, tame, perm, 1, R, F32), exact(x, sx, w, sw, tame, tame_p, 1, R), F32)


@pytest.mark.parametrize("R", [9, 300])
def test_gathered_rows_of_one_matrix(R):
    """A permutation without offsets: E = 1."""
    K, N, T = 208, 264, 7
    x, w, sx, sw = codes((T, K), 1), codes((1, N, K), 2), scales((T,), 3), scales((1, N), 4)
    perm = torch.randint(0, 3 * T, (R,), dtype=torch.int32, device="cuda", generator=torch.Generator("cuda").manual_seed(R))
    check(run(x, sx, w, sw, None, perm, 3, R, BF16), exact(x, sx, w, sw, None, perm, 3, R), BF16)


@pytest.mark.parametrize("E", [64, 63])
def test_many_experts_with_wild_offsets(E):
    """Every entry of the offsets counts, the last of 65 included, and none is trusted."""
    K, N, R = 64, 40, 500
    x, w, sx, sw = codes((R, K), 1), codes((E, N, K), 2), scales((R,), 3), scales((E, N), 4)
    g = np.random.default_rng(E)
    off = g.integers(-100, R + 100, E + 1).astype(np.int32)
    tame = np.maximum.accumulate(np.clip(off, 0, R))
    check(run(x, sx, w, sw, torch.from_numpy(off).cuda(), None, 1, R, F32),
          exact(x, sx, w, sw, torch.from_numpy(tame), None, 1, R), F32)
    off = np.sort(g.integers(0, R + 1, E + 1)).astype(np.int32)
    check(run(x, sx, w, sw, torch.from_numpy(off).cuda(), None, 1, R, F32),
          exact(x, sx, w, sw, torch.from_numpy(off), None, 1, R), F32)


def test_same_token_twice():
    """A token sent to several experts, and twice to one."""
    K, N = 192, 72
    x, w, sx, sw = codes((2, K), 1), codes((2, N, K), 2), scales((2,), 3), scales((2, N), 4)
    perm = torch.tensor([0, 1, 2, 3, 0, 2], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
    check(run(x, sx, w, sw, offsets, perm, 2, 6, BF16), exact(x, sx, w, sw, offsets, perm, 2, 6), BF16)


def test_offsets_past_32_bits():
    K, N, E = 8192, 40960, 16  # 5.4 GB of weights
    w = codes((E, N, K), 5)
    sw = scales((E, N), 6)
    c = [0] * (E - 2) + [3, 70]
    offsets, perm, T, rows = grouped(c, 1, 1)
    x, sx = codes((T, K), 7), scales((T,), 8)
    y = run(x, sx, w, sw, offsets, perm, 1, rows, BF16)
    check(y, exact(x, sx, w, sw, offsets, perm, 1, rows), BF16)
    del w, y
    K, N, T = 4096, 264, 1_100_000  # 4.5 GB of tokens, a few of them used
    x = torch.zeros(T, K, dtype=torch.int8, device="cuda")
    use = torch.tensor([0, 1, 524_287, 524_288, 1_048_575, 1_048_576, T - 2, T - 1], device="cuda")
    x[use] = codes((len(use), K), 9)
    w, sx, sw = codes((2, N, K), 10), scales((T,), 11), scales((2, N), 12)
    for rows in (8, 400):  # few rows, and a tile
        perm = use.repeat((rows + 7) // 8)[:rows].to(torch.int32)
        offsets = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
        y = run(x, sx, w, sw, offsets, perm, 1, rows, F32)
        check(y, exact(x, sx, w, sw, offsets, perm, 1, rows), F32)
    del x, w, y
    K, N, R = 64, 32768, 70000  # 2.3e9 outputs
    x, w, sx, sw = codes((R, K), 1), codes((1, N, K), 2), scales((R,), 3), scales((1, N), 4)
    y = torch.empty(R, N, dtype=BF16, device="cuda")
    M.moe_matmul_i8(x, sx, w, sw, None, None, R, 1, R, K, N, 1, y, M.MOE_BF16)
    pick = torch.tensor([0, 1, 65535, 65537, R - 2, R - 1], device="cuda")
    check(y[pick], exact(x[pick], sx[pick], w, sw, None, None, 1, len(pick)), BF16)


def test_quantize_codes():
    for T, m in [(1, 64), (5, 256), (33, 4096)]:
        g = torch.Generator().manual_seed(m)
        x = (torch.randn(T, m, generator=g) * torch.logspace(-20, 20, T)[:, None]).to(BF16).cuda()
        x[0] = 0
        c, s = torch.empty(T, m, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        M.moe_quantize_codes_i8(x, T, m, c, s)
        v, s2 = torch.empty_like(x), torch.empty_like(s)
        M.moe_quantize_rows_i8(x, T, m, v, s2)
        assert torch.equal(s, s2) and torch.equal((c.double() * s.double()[:, None]), v.double())
        _, codes_o, scales_o = oracle.quant_rows_i8(x.view(torch.int16).cpu().numpy().view(np.uint16))
        assert np.array_equal(c.cpu().numpy(), codes_o) and np.array_equal(s.cpu().numpy(), scales_o)


# 128 MB of weights or more, which are read as not to be kept where an expert
# has one row block: every tile shape, with experts of none, one and several
# row blocks; the last two with weights off their 128-byte lines
LARGE = {"t32x256": ([10, 0, 40, 3, 1, 9, 70, 8], 1024, 16392), "t64x64": ([30, 64, 0, 65, 1, 100, 17, 9], 8192, 2056),
         "t64x128": ([40, 64, 65, 0, 30, 1, 100, 32], 2048, 8200), "t128x256": ([90, 128, 129, 0, 64, 20, 200, 33], 2048, 8200),
         "t256x256": ([150, 256, 257, 0, 128, 100, 300, 33], 2048, 8200),
         "t128x128": ([100, 128, 0, 129, 5, 160, 90, 64] * 2, 4096, 2056), "r16": ([11], 16384, 8200), "r32": ([30], 16384, 8200),
         "r64": ([60], 16384, 8200), "r64_two_blocks": ([70], 16384, 8200),
         "r16_two_blocks": ([20, 2], 16384, 4104), "short_lines": ([10, 0, 40, 3, 1, 9, 70, 8], 1040, 16392),
         "shifted": ([10, 0, 40, 3, 1, 9, 70, 8], 1024, 16392)}


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", LARGE)
def test_large_weights(name, out):
    counts, K, N = LARGE[name]
    E, rows = len(counts), sum(counts)
    log(f"matmul_i8 large weights {name} E={E} K={K} N={N} {out}")
    w = codes((E * N * K + 128,), N)
    at = 16 if name == "shifted" else 0
    w = w[at:at + E * N * K].view(E, N, K)
    assert E * N * K >= 1 << 27
    offsets, perm, T, _ = grouped(counts, 2, E)
    x, sx, sw = codes((T, K), K), scales((T,), 1), scales((E, N), 2)
    if E == 1:
        x, sx, offsets, perm = codes((rows, K), K), scales((rows,), 1), None, None
    check(run(x, sx, w, sw, offsets, perm, 2, rows, out), exact(x, sx, w, sw, offsets, perm, 2, rows), out, "y")


# private rings of 16, 32 and 64 rows, one and more row blocks, partial last stages
PRIVATE = [(60, 272, 6168), (64, 2064, 6152), (100, 2064, 4104), (33, 4096, 7000), (130, 144, 2056), (20, 528, 4104),
           (32, 16, 8200), (16, 2064, 4104)]


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,K,N", PRIVATE)
def test_private_rings(R, K, N, out):
    log(f"matmul_i8 private rings R={R} K={K} N={N} {out}")
    x, w, sx, sw = codes((R, K), R + K), codes((1, N, K), N), scales((R,), 1), scales((1, N), 2)
    check(run(x, sx, w, sw, None, None, 1, R, out), exact(x, sx, w, sw, None, None, 1, R), out, "y")


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts,K,N", [([60, 0, 33, 70], 272, 2056), ([40, 100, 1, 20], 2064, 2056), ([33, 40], 2048, 4104)])
def test_private_rings_of_experts(counts, K, N, out):
    log(f"matmul_i8 private rings {counts} K={K} N={N} {out}")
    E = len(counts)
    offsets, perm, T, rows = grouped(counts, 2, E)
    x, w, sx, sw = codes((T, K), K), codes((E, N, K), N), scales((T,), 1), scales((E, N), 2)
    check(run(x, sx, w, sw, offsets, perm, 2, rows, out), exact(x, sx, w, sw, offsets, perm, 2, rows), out, "y")


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("K", [16, 272, 384, 1040, 4096])
@pytest.mark.parametrize("E,N", [(8, 5128), (1, 41000)])
def test_few_rows_of_wide_tiles(E, N, K, out):
    """One round of 32 x 256 tiles, with one to many stages and a partial last one."""
    counts = [10, 0, 40, 3, 1, 9, 70, 8] if E == 8 else [17]
    log(f"matmul_i8 wide tiles {counts} K={K} N={N} {out}")
    offsets, perm, T, rows = grouped(counts, 2, E)
    x, w, sx, sw = codes((T, K), K), codes((E, N, K), N), scales((T,), 1), scales((E, N), 2)
    check(run(x, sx, w, sw, offsets, perm, 2, rows, out), exact(x, sx, w, sw, offsets, perm, 2, rows), out, "y")


# 64 x 256 tiles: experts that mostly fit one block, one and two workgroups a CU
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("K", [16, 272, 1280, 2064])
@pytest.mark.parametrize("counts,N", [([40, 64, 0, 33, 1, 70, 100, 17], 14344), ([40, 64, 0, 33, 1, 70, 100, 17], 6152), ([64], 41000),
                                      ([33], 98312)])
def test_mid_rows_of_wide_tiles(counts, N, K, out):
    log(f"matmul_i8 wide tiles {counts} K={K} N={N} {out}")
    E = len(counts)
    offsets, perm, T, rows = grouped(counts, 2, E)
    x, w, sx, sw = codes((T, K), K), codes((E, N, K), N), scales((T,), 1), scales((E, N), 2)
    check(run(x, sx, w, sw, offsets, perm, 2, rows, out), exact(x, sx, w, sw, offsets, perm, 2, rows), out, "y")
