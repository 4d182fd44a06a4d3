"""The permute and the combine with the widest rows that an int counts, 2^31 - 8
columns: rows of zeros and ones with a few other columns, so that every sum
and product is exact."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

pytestmark = pytest.mark.gpu

m = 2**31 - 8
COLS = [0, 7, 511, 512, 2**30 - 8, 2**30, m - 2049, m - 513, m - 9, m - 8, m - 1]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def row(n, dtype, base, value):
    t = torch.full((n, m), base, dtype=dtype, device="cuda")
    t[:, COLS] = value
    return t


def is_row(t, base, value):
    assert t[COLS].tolist() == [value] * len(COLS)
    t[COLS] = base
    return float(t.amin()) == base and float(t.amax()) == base


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_widest_rows(dtype):
    code = M.MOE_BF16 if dtype == torch.bfloat16 else M.MOE_F32
    es = 2 if dtype == torch.bfloat16 else 4
    if torch.cuda.mem_get_info()[0] < 8 * m * es:
        pytest.skip("needs eight such rows")
    inv = torch.tensor([1, 0], dtype=torch.int32, device="cuda")  # one token of two rows
    w = torch.tensor([[2.0, 4.0]], device="cuda")
    x = row(1, dtype, 1.0, 3.0)
    xp = torch.zeros(2, m, dtype=dtype, device="cuda")
    print(f"permute {dtype}", flush=True)
    M.moe_permute_rows(x, code, inv, 1, m, 2, 2, xp)
    assert is_row(xp[0], 1.0, 3.0) and is_row(xp[1], 1.0, 3.0)
    del xp

    yp = row(2, dtype, 0.0, 1.0)
    yp[1, COLS] = 2.0
    print(f"combine {dtype}", flush=True)
    y = torch.empty(1, m, dtype=dtype, device="cuda")
    M.moe_combine_rows(yp, code, inv, w, 1, m, 2, 2, y, code)
    assert is_row(y[0], 0.0, 8.0)  # 2 * 2 + 4 * 1
    M.moe_permute_rows_backward(yp, code, inv, 1, m, 2, 2, y, code)
    assert is_row(y[0], 0.0, 3.0)
    del y

    print(f"combine backward {dtype}", flush=True)
    dyp = torch.zeros(2, m, dtype=dtype, device="cuda")
    dw = torch.empty(1, 2, device="cuda")
    M.moe_combine_rows_backward(x, code, yp, code, inv, w, 1, m, 2, 2, dyp, dw)
    assert dw.tolist() == [[6.0 * len(COLS), 3.0 * len(COLS)]]
    assert is_row(dyp[1], 2.0, 6.0) and is_row(dyp[0], 4.0, 12.0)
