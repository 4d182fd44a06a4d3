"""Every kernel of the int8 product, on sizes that select it, against the
definition in 64 bits (bounds as in test_gpu_matmul_i8)."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

from _gpu import log
from _i8_tiles import CASES
from test_gpu_matmul_i8 import BF16, F32, check, codes, exact, grouped, run, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", CASES)
def test_kernel(name, out):
    counts, K, N, kernel, _, kept_out = CASES[name]
    E, rows, k = len(counts), sum(counts), 2
    log(f"matmul_i8 {name}: {kernel}, rows {counts} K={K} N={N} {out}")
    w, sw = codes((E, N, K), N), scales((E, N), 2)
    assert w.data_ptr() % 128 == 0 and (not kept_out or (K % 128 == 0 and E * N * K >= 1 << 27))
    offsets, perm, T, _ = grouped(counts, k, E)
    if E == 1:
        offsets, perm, T, k = None, None, rows, 1
    x, sx = codes((T, K), K), scales((T,), 1)
    check(run(x, sx, w, sw, offsets, perm, k, rows, out), exact(x, sx, w, sw, offsets, perm, k, rows), out, "y")
