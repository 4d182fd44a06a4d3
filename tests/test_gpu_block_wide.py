"""The trainable block's operators on tensors of more than 2^31 elements: what lies past 32-bit
offsets against 64-bit definitions of those rows (or that expert) alone."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

import _block
from _gpu import log

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def rnd(*s, seed=0, scale=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*s, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def test_gated_rows():
    """140000 rows of 16384: gate, up and the hidden rows pass 2^31 elements."""
    R, m, p, tail = 140000, 64, 16384, 300
    log(f"gated rows {R} x {p}")
    x, dy = rnd(R, m, seed=1), rnd(R, m, seed=2)
    wg, wu, wd = (rnd(1, *s, seed=i, scale=s[0] ** -0.5) for i, s in ((3, (m, p)), (4, (m, p)), (5, (p, m))))
    y, gate, up = (torch.empty(R, n, dtype=BF16, device="cuda") for n in (m, p, p))
    n = M.moe_gated_ffn_workspace_size(M.MOE_BF16, R, m, p, 1, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    M.moe_gated_ffn_forward(x, M.MOE_BF16, wg, wu, wd, None, None, R, 1, R, m, p, 1, y, gate, up, ws, n)
    dx = torch.empty_like(y)
    M.moe_gated_ffn_backward(dy, x, M.MOE_BF16, wg, wu, wd, gate, up, None, None, R, 1, R, m, p, 1, dx, None, None, None, ws, n)
    torch.cuda.synchronize()
    want, bound = _block.forward(x[-tail:], wg, wu, wd, None, None, 1, tail, BF16)
    for name, o, w, b in zip(("y", "gate", "up"), (y, gate, up), want, bound):
        _block.check(o[-tail:], w, b, name, log)
    want, bound = _block.backward(dy[-tail:], x[-tail:], wg, wu, wd, gate[-tail:], up[-tail:], None, None, 1, tail, BF16)
    _block.check(dx[-tail:], want[0], bound[0], "dx", log)


def test_gated_experts():
    """64 experts of 8192 x 4104: weights and their gradients pass 2^31 elements."""
    E, m, p, R = 64, 8192, 4104, 130
    log(f"gated experts {E} x {m} x {p}")
    x, dy = rnd(R, m, seed=1), rnd(R, m, seed=2)
    wg, wu, wd = (torch.zeros(E, *s, dtype=BF16, device="cuda") for s in ((m, p), (m, p), (p, m)))
    for i, w in enumerate((wg, wu, wd)):
        w[-1] = rnd(*w.shape[1:], seed=3 + i, scale=w.shape[1] ** -0.5)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = R
    y, gate, up = (torch.empty(R, n, dtype=BF16, device="cuda") for n in (m, p, p))
    n = M.moe_gated_ffn_workspace_size(M.MOE_BF16, R, m, p, E, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    M.moe_gated_ffn_forward(x, M.MOE_BF16, wg, wu, wd, off, None, R, 1, R, m, p, E, y, gate, up, ws, n)
    dx = torch.empty_like(y)
    dw = [torch.full_like(w, 3.0) for w in (wg, wu, wd)]
    M.moe_gated_ffn_backward(dy, x, M.MOE_BF16, wg, wu, wd, gate, up, off, None, R, 1, R, m, p, E, dx, *dw, ws, n)
    torch.cuda.synchronize()
    one = [w[-1:] for w in (wg, wu, wd)]
    want, bound = _block.forward(x, *one, None, None, 1, R, BF16)
    for name, o, w, b in zip(("y", "gate", "up"), (y, gate, up), want, bound):
        _block.check(o, w, b, name, log)
    want, bound = _block.backward(dy, x, *one, gate, up, None, None, 1, R, BF16)
    for name, o, w, b in zip(("dx", "dw_gate", "dw_up", "dw_down"), [dx] + [t[-1:] for t in dw], want, bound):
        _block.check(o, w, b, name, log)
    assert all(not bool(t[:-1].any()) for t in dw)


def test_add_norm():
    T, m, tail = 270000, 8192, 100
    log(f"add norm {T} x {m}")
    x, r, gamma = rnd(T, m, seed=1), rnd(T, m, seed=2), 1 + rnd(m, seed=3, scale=0.1, dtype=F32)
    s, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    codes, scale = torch.empty(T, m, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    M.moe_add_norm_forward(x, r, M.MOE_BF16, M.MOE_NORM_RMS, gamma, None, 1e-5, T, m, s, y, codes, scale, None, rstd)
    few = [torch.empty_like(t[-tail:]) for t in (s, y, codes, scale, rstd)]
    M.moe_add_norm_forward(x[-tail:], r[-tail:], M.MOE_BF16, M.MOE_NORM_RMS, gamma, None, 1e-5, tail, m, few[0], few[1], few[2],
                           few[3], None, few[4])
    # (a call that moves this much reads its inputs past the caches: another kernel, the same arithmetic)
    for a, b, name in zip((s, y, codes, scale, rstd), few, ("sum", "y", "codes", "scale", "rstd")):
        assert torch.equal(a[-tail:], b), name
    dx, one = torch.empty_like(x), torch.empty_like(few[0])
    M.moe_add_norm_backward(x, r, s, M.MOE_BF16, M.MOE_NORM_RMS, gamma, None, rstd, T, m, dx, None, None)
    M.moe_add_norm_backward(x[-tail:], r[-tail:], s[-tail:], M.MOE_BF16, M.MOE_NORM_RMS, gamma, None, few[4], tail, m, one, None, None)
    assert torch.equal(dx[-tail:], one)


def test_route():
    T, m, E, k, tail = 540000, 4096, 8, 2, 200
    log(f"route gradient {T} x {m}")
    g = torch.Generator(device="cuda").manual_seed(4)
    x, add = rnd(T, m, seed=1), rnd(T, m, seed=2)
    idx = torch.topk(torch.rand(T, E, generator=g, device="cuda"), k).indices.to(torch.int32)
    w = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
    dw = torch.randn(T, k, generator=g, device="cuda")
    wr = rnd(m, E, seed=3, scale=m**-0.5, dtype=F32)
    dl, dx, dwr, db = torch.empty(T, E, device="cuda"), torch.empty_like(x), torch.empty(m, E, device="cuda"), torch.empty(E, device="cuda")
    n = M.moe_route_backward_workspace_size(T, m, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    M.moe_route_backward(dw, idx, w, None, x, M.MOE_BF16, wr, add, T, m, E, k, dl, dx, dwr, db, ws, n)
    torch.cuda.synchronize()
    e = slice(T - tail, T)
    want, bound = _block.route_backward(dw[e], idx[e], w[e], None, x[e], wr, add[e], E, BF16)
    _block.check(dl[e], want[0], bound[0], "d_logits", log)
    _block.check(dx[e], want[1], bound[1], "dx", log)
    total, size = torch.zeros(m, E, dtype=torch.float64, device="cuda"), torch.zeros(m, E, dtype=torch.float64, device="cuda")
    for a in range(0, T, 60000):
        c, d = x[a:a + 60000].double(), dl[a:a + 60000].double()
        total += c.T @ d
        size += c.abs().T @ d.abs()
    _block.check(dwr, total, 2 * (T + 1) * 2.0**-24 * size, "dw_router", log)
