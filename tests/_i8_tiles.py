"""Sizes for every kernel of the int8 product: {name: (rows of each expert, K,
N, kernel, once, kept out of the caches)}, the kernel being the one that the
rule picks on 256 CUs (tests/test_i8_choice.py holds it to that).  Each has
more stages than its ring, most a partial last one; the experts' row counts lie around the
mean, with experts of none and of several row blocks."""

AROUND = {16: [10, 0, 40, 3, 1, 9, 57, 8], 20: [30, 64, 0, 5, 1, 30, 17, 9], 40: [40, 64, 0, 33, 1, 70, 100, 17],
          44: [40, 64, 65, 0, 30, 1, 100, 52], 90: [90, 128, 129, 0, 64, 20, 200, 89],
          150: [150, 256, 257, 0, 128, 100, 276, 33], 300: [300, 257, 1, 512, 700, 0, 255, 375]}

CASES = {
    # (tiles of 32 and 64 rows by 256 channels, one workgroup a CU with three stages, two with two)
    "32x256x3": (AROUND[16], 816, 5128, "32x256x3", True, False),
    "32x256x3_dense": ([17], 816, 41000, "32x256x3", True, False),
    "32x256x3_large": (AROUND[16], 3328, 5128, "32x256x3", True, True),
    "32x256x3_large_dense": ([17], 3328, 41000, "32x256x3", True, True),
    "64x256x3": (AROUND[40], 816, 5128, "64x256x3", True, False),
    "64x256x3_large": (AROUND[40], 3328, 5128, "64x256x3", True, True),
    "32x256x2": (AROUND[16], 816, 14328, "32x256x2", True, False),
    "32x256x2_large": (AROUND[16], 1280, 14328, "32x256x2", True, True),
    "32x256x2_large_dense": ([32], 1152, 130000, "32x256x2", True, True),
    "64x256x2": (AROUND[40], 816, 14328, "64x256x2", True, False),
    "64x256x2_large": (AROUND[40], 1280, 14328, "64x256x2", True, True),
    "256x256": (AROUND[300], 560, 4104, "256x256x2", False, False),
    "256x256_once": (AROUND[150], 560, 8200, "256x256x2", True, False),
    "256x256_large": (AROUND[150], 2176, 8200, "256x256x2", True, True),
    "256x256_large_shared": (AROUND[300], 2176, 8200, "256x256x2", False, False),
    "128x256": ([150, 129, 256, 0, 257, 200, 100, 33], 688, 3080, "128x256x3", False, False),
    "128x256_once": (AROUND[90], 688, 8200, "128x256x3", True, False),
    "128x256_large": (AROUND[90], 2176, 8200, "128x256x3", True, True),
    "128x128": ([300], 816, 8200, "128x128x4", False, False),
    "128x128_once": (AROUND[90] * 2, 816, 1800, "128x128x4", True, False),
    "128x128_large": (AROUND[90] * 2, 4736, 1800, "128x128x4", True, True),
    "64x128": ([515], 816, 4008, "64x128x3", False, False),
    "64x128_once": (AROUND[44], 816, 3336, "64x128x3", True, False),
    "64x128_large": (AROUND[44], 5120, 3336, "64x128x3", True, True),
    "64x64": ([70], 816, 8200, "64x64x4", False, False),
    "64x64_once": (AROUND[20], 816, 2056, "64x64x4", True, False),
    "64x64_large": (AROUND[20], 8192, 2056, "64x64x4", True, True),
    # (private rings of four waves: the reduction split over them)
    "ring16": ([17, 3, 0, 40, 1, 16, 9, 5], 2064, 1032, "ring16", True, False),
    "ring16_large": ([11], 16384, 8200, "ring16", True, True),
    "ring16_large_experts": ([20, 2, 0, 15], 16512, 2056, "ring16", True, True),
    "ring64": ([60], 4112, 8200, "ring64", True, False),
    "ring64_experts": ([60, 0, 33, 70], 2064, 2056, "ring64", True, False),
    "ring64_large": ([60], 16512, 8200, "ring64", True, True),
    "ring64_large_experts": ([60, 70, 33, 1], 16384, 2056, "ring64", True, True),
    "ring32": ([20], 4112, 8200, "ring32", True, False),
    "ring32_experts": ([33, 0, 70, 20], 2064, 1032, "ring32", True, False),
    "ring32_large": ([30], 16512, 8200, "ring32", True, True),
    "ring32_large_experts": ([30, 40, 1, 20], 16384, 2056, "ring32", True, True),
}
