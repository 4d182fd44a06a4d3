"""Parts of the residual norm's gradient: each output without the others, with and without dsum."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

from test_gpu_add_norm import BF16, CODE, F32, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,m", [(1, 64), (5, 72), (1100, 264), (777, 5000), (300, 9000)])
def test_outputs_alone(T, m, dtype):
    """dsum reaches dx alone: dgamma and dbeta have the same bits without it, without dx, and where it holds NaN."""
    s, dy, ds = rnd((T, m), dtype, 1, 2.0, 0.5), rnd((T, m), dtype, 2), rnd((T, m), dtype, 3)
    gamma, mean, rstd = rnd((m,), F32, 4, 0.2, 1.0), rnd((T,), F32, 5, 0.3), rnd((T,), F32, 6, 0.0, 0.5)
    n = M.moe_norm_backward_workspace_size(T, m)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")

    def call(dsum, *wanted):
        o = dict(dx=torch.full_like(s, 7), dgamma=torch.full_like(gamma, 7), dbeta=torch.full_like(gamma, 7))
        a = {name: t if name in wanted else None for name, t in o.items()}
        M.moe_add_norm_backward(dy, dsum, s, CODE[dtype], M.MOE_NORM_LAYER, gamma, mean, rstd, T, m, a["dx"], a["dgamma"],
                                a["dbeta"], ws, n)
        return o

    full = call(ds, "dx", "dgamma", "dbeta")
    nan = torch.full_like(ds, float("nan"))
    for dsum in (ds, None, nan):
        for wanted in (("dgamma", "dbeta"), ("dgamma",), ("dbeta",)):
            got = call(dsum, *wanted)
            assert all(torch.equal(got[name], full[name]) for name in wanted), wanted
            assert all(bool((got[name] == 7).all()) for name in got if name not in wanted), wanted
    assert torch.equal(call(ds, "dx")["dx"], full["dx"])
