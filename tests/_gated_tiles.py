"""Sizes for every kernel of the gated feed-forward block: {name: (bf16, rows, m, p, experts)}.
KERNELS lists the kernels that the choice rules take on 256 CUs as (type, product, tile, weights
kept in the caches or "once", whole or "split" reductions, rows in "two" parts or one), and
tests/test_gated_choice.py holds the sizes to covering each with more stages than its ring."""
import random

PRODUCTS = ("up", "down", "hidden", "x")  # gate and up, Y = H W_d, hidden gradients, dX


def offsets(rows, E):
    """The experts' row ranges: cut anywhere, so that some experts take several times the mean, one (of
    four or more) none; of thirty rows or more one before and two behind belong to no expert."""
    g = random.Random(rows * 131 + E)
    lo, hi = (1, rows - 2) if rows >= 30 and E > 1 else (0, rows)
    cuts = sorted(g.randint(lo, hi) for _ in range(E - 1))
    if E >= 4:
        cuts[1] = cuts[0]
    return [lo, *cuts, hi]


def most(rows, E):
    """Rows of the fullest expert."""
    o = offsets(rows, E)
    return max(b - a for a, b in zip(o, o[1:]))


_BF16 = [("256x256x2", "kept", "whole"), ("128x256x3", "kept", "whole"),
         *((t, "kept", s) for t in ("128x128x2", "64x128x3", "32x256x3") for s in ("whole", "split")),
         ("32x256x2", "kept", "whole"), ("32x256x2", "once", "whole"), ("32x256x3", "once", "whole"), ("32x256x3", "once", "split")]
_F32 = [(t, "kept", s) for t in ("128x128x2", "64x128x3", "32x128x2") for s in ("whole", "split")]
KERNELS = {("bf16", op, *t, "two" if t[0].startswith("32") and op in ("down", "x") else "one") for op in PRODUCTS for t in _BF16}
KERNELS |= {("f32", op, *t, "one") for op in PRODUCTS for t in _F32}
KERNELS |= {("bf16", "w", "256x256x2", "kept", "whole", n) for n in ("one", "two")}
KERNELS |= {("bf16", "w", "128x128x2", "kept", s, n) for s, n in (("whole", "one"), ("split", "one"), ("whole", "two"))}
KERNELS |= {("f32", "w", "128x128x2", "kept", s, "one") for s in ("whole", "split")}

CASES = {
    "bf16_11_rows_5_experts_2536_5264": (True, 11, 2536, 5264, 5),
    "bf16_16_rows_16_experts_4904_432": (True, 16, 4904, 432, 16),
    "bf16_34_rows_33_experts_1680_1200": (True, 34, 1680, 1200, 33),
    "bf16_42_rows_33_experts_1808_80": (True, 42, 1808, 80, 33),
    "bf16_46_rows_33_experts_144_1872": (True, 46, 144, 1872, 33),
    "bf16_75_rows_2_experts_984_72": (True, 75, 984, 72, 2),
    "bf16_78_rows_2_experts_24_1000": (True, 78, 24, 1000, 2),
    "bf16_103_rows_5_experts_232_248": (True, 103, 232, 248, 5),
    "bf16_109_rows_7_experts_1120_1080": (True, 109, 1120, 1080, 7),
    "bf16_178_rows_2_experts_136_160": (True, 178, 136, 160, 2),
    "bf16_241_rows_64_experts_1056_1192": (True, 241, 1056, 1192, 64),
    "bf16_1699_rows_33_experts_264_616": (True, 1699, 264, 616, 33),
    "bf16_2973_rows_2_experts_1824_208": (True, 2973, 1824, 208, 2),
    "bf16_4107_rows_3_experts_200_1296": (True, 4107, 200, 1296, 3),
    "bf16_8470_rows_33_experts_144_528": (True, 8470, 144, 528, 33),
    "bf16_8964_rows_33_experts_528_168": (True, 8964, 528, 168, 33),
    "f32_75_rows_2_experts_80_80": (False, 75, 80, 80, 2),
    "f32_491_rows_2_experts_272_288": (False, 491, 272, 288, 2),
    "f32_646_rows_2_experts_944_528": (False, 646, 944, 528, 2),
    "f32_1548_rows_3_experts_840_536": (False, 1548, 840, 536, 3),
    "f32_8434_rows_7_experts_696_656": (False, 8434, 696, 656, 7),
    "f32_8495_rows_64_experts_144_152": (False, 8495, 144, 152, 64),
}
