"""Sums over the rows of tensors of more than 2^31 elements.  Only a few hundred rows give terms that
are not zero, on both sides of element 2^31 and at the end: adding zeros is exact, so the bounds count
those rows alone, and a row that is lost or read elsewhere stands out."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

import _block
from _gpu import log
from test_gpu_block_wide import BF16, F32, rnd

pytestmark = pytest.mark.gpu

u = 2.0**-24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def some_rows(rows, columns):
    """The first rows, those around element 2^31, and the last."""
    at = (1 << 31) // columns
    assert 200 < at - 60 and at + 60 < rows - 200
    return torch.cat([torch.arange(100), torch.arange(at - 50, at + 50), torch.arange(rows - 200, rows)]).cuda()


def only(t, keep):
    """t with zeros in all other rows."""
    out = torch.zeros_like(t)
    out[keep] = t[keep]
    return out


def counts(got, want, bound, what):
    """Within the bound, which is far below the values themselves."""
    _block.check(got, want, bound, what, log)
    assert float(want.abs().max()) > 100 * float(bound.max()), what


def test_route():
    T, m, E, k = 540000, 4096, 8, 2
    log(f"route gradient's sums over {T} x {m}")
    keep = some_rows(T, m)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = rnd(T, m, seed=1)
    idx = torch.topk(torch.rand(T, E, generator=g, device="cuda"), k).indices.to(torch.int32)
    w = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
    dw = only(torch.randn(T, k, generator=g, device="cuda"), keep)  # dw = 0: d_logits = 0
    wr = rnd(m, E, seed=3, scale=m**-0.5, dtype=F32)
    dl, dx = torch.empty(T, E, device="cuda"), torch.empty_like(x)
    dwr, db = torch.empty(m, E, device="cuda"), torch.empty(E, device="cuda")
    n = M.moe_route_backward_workspace_size(T, m, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    M.moe_route_backward(dw, idx, w, None, x, M.MOE_BF16, wr, None, T, m, E, k, dl, dx, dwr, db, ws, n)
    torch.cuda.synchronize()
    want, bound = _block.route_backward(dw[keep], idx[keep], w[keep], None, x[keep], wr, None, E, BF16)
    _block.check(dl[keep], want[0], bound[0], "d_logits", log)
    _block.check(dx[keep], want[1], bound[1], "dx", log)
    counts(dwr, want[2], bound[2], "dw_router")
    counts(db, want[3], bound[3], "db_router")
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[keep] = False
    assert not bool(dl[rest].any())


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_add_norm(norm):
    T, m, layer = 270000, 8192, norm == "layer"
    log(f"residual norm's sums over {T} x {m}, {norm}")
    keep = some_rows(T, m)
    x, r, gamma = rnd(T, m, seed=1, scale=0.5), rnd(T, m, seed=2), 1 + rnd(m, seed=3, scale=0.1, dtype=F32)
    s, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda") if layer else None, torch.empty(T, device="cuda")
    kind = M.MOE_NORM_LAYER if layer else M.MOE_NORM_RMS
    M.moe_add_norm_forward(x, r, M.MOE_BF16, kind, gamma, None, 1e-5, T, m, s, x, None, None, mean, rstd)
    dy = only(r, keep)
    dgamma, dbeta = torch.empty(m, device="cuda"), torch.empty(m, device="cuda") if layer else None
    n = M.moe_norm_backward_workspace_size(T, m)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    M.moe_add_norm_backward(dy, r, s, M.MOE_BF16, kind, gamma, mean, rstd, T, m, None, dgamma, dbeta, ws, n)
    torch.cuda.synchronize()
    d, h = dy[keep].double(), s[keep].double()
    h = (h - mean[keep].double()[:, None] if layer else h) * rstd[keep].double()[:, None]
    # the deviation, the product with rstd and with dy round once each, an addition for every term
    counts(dgamma, (d * h).sum(0), (len(keep) + 6) * u * (d * h).abs().sum(0), "dgamma")
    if layer:
        counts(dbeta, d.sum(0), (len(keep) + 3) * u * d.abs().sum(0), "dbeta")


def test_gated_weights():
    """140000 rows of 16384: the hidden rows' gradients and the hidden rows pass 2^31 elements."""
    R, m, p = 140000, 64, 16384
    log(f"gated weight gradients over {R} x {p}")
    keep = some_rows(R, p)
    x, dy = rnd(R, m, seed=1), only(rnd(R, m, seed=2), keep)
    wg, wu, wd = (rnd(1, *s, seed=i, scale=s[0]**-0.5) for i, s in ((3, (m, p)), (4, (m, p)), (5, (p, m))))
    gate, up = rnd(R, p, seed=6), rnd(R, p, seed=7)
    dw = [torch.empty_like(w) for w in (wg, wu, wd)]
    n = M.moe_gated_ffn_workspace_size(M.MOE_BF16, R, m, p, 1, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    M.moe_gated_ffn_backward(dy, x, M.MOE_BF16, wg, wu, wd, gate, up, None, None, R, 1, R, m, p, 1, None, *dw, ws, n)
    torch.cuda.synchronize()
    want, bound = _block.backward(dy[keep], x[keep], wg, wu, wd, gate[keep], up[keep], None, None, 1, len(keep), BF16)
    for name, o, w, b in zip(("dw_gate", "dw_up", "dw_down"), dw, want[1:], bound[1:]):
        _block.check(o, w, b, name, log)
