"""The combine's gradient written over the rows it reads (dy_perm = y_perm):
the bits of the call with separate buffers."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

from test_gpu_rows import CODE, F32, PAIRS, ROW_CASES, ids, plan, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


# the cases of the operator's own test, and one that moves more than 128 MB
@pytest.mark.parametrize("pair", PAIRS, ids=ids)
@pytest.mark.parametrize("T,k,E,m,drop", ROW_CASES + [(4096, 2, 8, 4104, 0.1)])
def test_combine_backward_in_place(T, k, E, m, drop, pair):
    rt, tt = pair
    inv, rows = plan(T, k, E, drop, T + m)
    r, dy, w = rnd((rows + 2, m), rt, m + 1), rnd((T, m), tt, m + 3), rnd((T, k), F32, m + 2)
    out, dw = r.clone(), torch.empty(T, k, device="cuda")
    M.moe_combine_rows_backward(dy, CODE[tt], r, CODE[rt], inv, w, T, m, k, rows, out, dw)
    here, dw_here = r.clone(), torch.empty_like(dw)
    M.moe_combine_rows_backward(dy, CODE[tt], here, CODE[rt], inv, w, T, m, k, rows, here, dw_here)
    assert torch.equal(here, out) and torch.equal(dw_here, dw)
    assert torch.equal(here[rows:], r[rows:])
