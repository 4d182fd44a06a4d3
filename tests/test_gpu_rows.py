"""The row operators around the experts (norm, permute, combine and their
gradients) against plain 64-bit implementations.

Every bound below is a count of roundings: u = 2^-24 is half an fp32 step,
U[dtype] half a step of the stored type.  A sum of n terms in any order is
within (n - 1) u sum|terms| of its exact value (first order), and each other
fp32 operation adds u of its result.  The bounds use the worst case over all
orders, so they hold whatever the kernels' split.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

from _gpu import log

pytestmark = pytest.mark.gpu

u = 2.0**-24
U = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8}
CODE = {torch.float32: M.MOE_F32, torch.bfloat16: M.MOE_BF16}
F32, BF16 = torch.float32, torch.bfloat16
TINY = 1e-37  # results below the normal range round absolutely


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


def rnd(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).cuda()


def n64(t):
    return None if t is None else t.double().cpu().numpy()


def check(got, ref, bar, what):
    got = n64(got)
    assert got.shape == ref.shape, what
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    err = np.abs(got - ref)
    bar = bar + TINY
    worst = float(np.max(err / bar)) if err.size else 0.0
    log(f"  {what}: max|err| {err.max() if err.size else 0:.3e}, {worst:.3f} of the bound")
    assert worst <= 1.0, what


class Guarded:
    """An output between two guard zones that must stay as they were."""

    def __init__(self, shape, dtype, fill=float("nan")):
        n = int(np.prod(shape))
        self.buf = torch.full((n + 128,), 7.0, dtype=dtype, device="cuda")
        self.t = self.buf[64:64 + n].view(shape)  # 64 elements: 16-byte aligned for both types
        self.t.fill_(fill)

    def intact(self):
        assert bool((self.buf[:64] == 7).all()) and bool((self.buf[64 + self.t.numel():] == 7).all())


# ---- norm -------------------------------------------------------------------------

NORM_SHAPES = [(1, 8), (3, 64), (5, 72), (1, 520), (7, 1000), (4, 2048), (3, 2056), (2, 4096), (6, 5000), (2, 8200),
               (3, 16384), (1100, 64), (2100, 2048), (700, 4104)]


def norm_ref(x, gamma, beta, eps, layer):
    mu = x.mean(1) if layer else np.zeros(len(x))
    d = x - mu[:, None]
    r = 1.0 / np.sqrt((d * d).mean(1) + eps)
    h = d * r[:, None]
    y = h * gamma + (beta if beta is not None else 0.0)
    return y, mu, r, h


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("norm", ["layer", "layer_nobeta", "rms"])
@pytest.mark.parametrize("T,m", NORM_SHAPES)
def test_norm_forward(T, m, norm, dtype):
    layer = norm != "rms"
    log(f"norm forward {norm} {dtype} T={T} m={m}")
    x = rnd((T, m), dtype, T * m, 2.0, 1.5)
    gamma, beta = rnd((m,), F32, 1, 0.2, 1.0), rnd((m,), F32, 2, 0.3) if norm == "layer" else None
    eps = 1e-5
    y, mean, rstd = Guarded((T, m), dtype), Guarded((T,), F32), Guarded((T,), F32)
    M.moe_norm_forward(x, CODE[dtype], M.MOE_NORM_LAYER if layer else M.MOE_NORM_RMS, gamma, beta, eps, T, m, y.t,
                       mean.t if layer else None, rstd.t)
    torch.cuda.synchronize()
    x64, g64, b64 = n64(x), n64(gamma), n64(beta)
    ref, mu, r, h = norm_ref(x64, g64, b64, eps, layer)
    avg = np.abs(x64).mean(1)
    e_mu = (m + 2) * u * avg if layer else np.zeros(T)  # the sum and its division
    # d = x - mu: e_mu and a rounding.  Sum of squares: relative (m + 4) u, and
    # mu's error shifts the sum of squares by m e_mu^2 only (the deviations sum to zero)
    e_r = 0.5 * ((m + 6) * u + (e_mu * r) ** 2) + 4 * u  # relative: half the sum's, square root, division
    check(rstd.t, r, r * e_r, "rstd")
    if layer:
        check(mean.t, mu, e_mu, "mean")
    e_h = (e_mu * r)[:, None] + np.abs(h) * (e_r[:, None] + 3 * u)
    bar = np.abs(g64) * e_h + 2 * u * np.abs(h * g64) + 2 * u * (np.abs(ref)) + U[dtype] * np.abs(ref)
    check(y.t, ref, bar * (1 + 2.0**-7), "y")
    for o in (y, mean, rstd):
        o.intact()


def test_norm_forward_leaves_statistics_out():
    x = rnd((5, 256), BF16, 3)
    g = rnd((256,), F32, 4, 0.1, 1)
    a, b = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    M.moe_norm_forward(x, M.MOE_BF16, M.MOE_NORM_LAYER, g, None, 1e-5, 5, 256, a)
    M.moe_norm_forward(x, M.MOE_BF16, M.MOE_NORM_LAYER, g, None, 1e-5, 5, 256, b, mean, rstd)
    assert torch.equal(a, b)


@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
def test_norm_special_rows(layer):
    """Constant, zero, huge, infinite and NaN rows: each row is its own, and a
    row's non-finite values do not reach the others."""
    m, eps = 512, 1e-6
    x = rnd((7, m), F32, 5)
    x[1] = 3.0
    x[2] = 0.0
    x[3] *= 1e15
    x[4, 17] = float("inf")
    x[5, 400] = float("nan")
    g = torch.ones(m, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(7, device="cuda")
    M.moe_norm_forward(x, M.MOE_F32, M.MOE_NORM_LAYER if layer else M.MOE_NORM_RMS, g, None, eps, 7, m, y, None, rstd)
    y64 = n64(y)
    ref, _, r, h = norm_ref(n64(x[[0, 1, 2, 3, 6]]), n64(g), None, eps, layer)
    bar = (m + 20) * u * (np.abs(ref) + (np.abs(n64(x[[0, 1, 2, 3, 6]])).mean(1) * r)[:, None])
    assert np.all(np.abs(y64[[0, 1, 2, 3, 6]] - ref) <= bar)
    assert np.all(y64[2] == 0.0)
    assert np.isnan(y64[4, 17]) and np.all(np.isnan(y64[5]))  # inf * 0 and NaN, as the formula gives


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("T,m", NORM_SHAPES + [(600, 16384)])
def test_norm_backward(T, m, layer, dtype):
    log(f"norm backward layer={layer} {dtype} T={T} m={m}")
    x, dy = rnd((T, m), dtype, T + m, 2.0, 0.7), rnd((T, m), dtype, T + 2 * m, 0.5, 0.1)
    gamma = rnd((m,), F32, 7, 0.3, 1.0)
    x64, dy64, g64 = n64(x), n64(dy), n64(gamma)
    _, mu, r, _ = norm_ref(x64, g64, None, 1e-5, layer)
    mean, rstd = torch.from_numpy(mu).float().cuda() if layer else None, torch.from_numpy(r).float().cuda()
    mu, r = n64(mean) if layer else np.zeros(T), n64(rstd)  # the operator's inputs are the fp32 values
    h = (x64 - mu[:, None]) * r[:, None]
    v = dy64 * g64
    s1, s2 = (v * h).mean(1, keepdims=True), v.mean(1, keepdims=True) if layer else np.zeros((T, 1))
    ref = (v - h * s1 - s2) * r[:, None]
    n = M.moe_norm_backward_workspace_size(T, m)
    ws = torch.full((n + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    dx, dg, db = Guarded((T, m), dtype), Guarded((m,), F32), Guarded((m,), F32)
    kind = M.MOE_NORM_LAYER if layer else M.MOE_NORM_RMS
    M.moe_norm_backward(dy, x, CODE[dtype], kind, gamma, mean, rstd, T, m, dx.t, dg.t, db.t if layer else None, ws, n)
    torch.cuda.synchronize()
    # h: two roundings; v: one; the averages: any-order sums of m terms of
    # three roundings each, one for the 1/m factor and one for the product
    e1 = (m + 6) * u * np.abs(v * h).mean(1, keepdims=True)
    e2 = (m + 4) * u * np.abs(v).mean(1, keepdims=True) if layer else 0.0
    parts = np.abs(v) + np.abs(h * s1) + np.abs(s2)
    bar = r[:, None] * (6 * u * parts + np.abs(h) * e1 + e2) + 2 * u * np.abs(ref) + U[dtype] * np.abs(ref)
    check(dx.t, ref, bar * (1 + 2.0**-7), "dx")
    check(dg.t, (dy64 * h).sum(0), (T + 4) * u * np.abs(dy64 * h).sum(0), "dgamma")
    if layer:
        check(db.t, dy64.sum(0), (T + 1) * u * np.abs(dy64).sum(0), "dbeta")
    for o in (dx, dg, db):
        o.intact()
    assert bool((ws[n:] == 0x5A).all())
    # each output alone has the same bits
    one = torch.empty_like(dx.t)
    M.moe_norm_backward(dy, x, CODE[dtype], kind, gamma, mean, rstd, T, m, one, None, None)
    assert torch.equal(one, dx.t)
    one = torch.empty_like(dg.t)
    M.moe_norm_backward(dy, x, CODE[dtype], kind, gamma, mean, rstd, T, m, None, one, None, ws, n)
    assert torch.equal(one, dg.t)
    if layer:
        M.moe_norm_backward(dy, x, CODE[dtype], kind, gamma, mean, rstd, T, m, None, None, one, ws, n)
        assert torch.equal(one, db.t)


def test_norm_without_eps_and_unaligned_refused():
    """eps 0 on rows that vary; a pointer off its 16 bytes is refused, not read."""
    T, m = 3, 264
    x, g = rnd((T, m), F32, 1, 3.0), rnd((m,), F32, 2, 0.1, 1.0)
    y = torch.empty_like(x)
    M.moe_norm_forward(x, M.MOE_F32, M.MOE_NORM_RMS, g, None, 0.0, T, m, y)
    ref = norm_ref(n64(x), n64(g), None, 0.0, False)[0]
    assert np.all(np.abs(n64(y) - ref) <= (m + 20) * u * np.abs(ref))
    off = torch.empty(T * m + 1, device="cuda")[1:].view(T, m)
    for args in [(off, g, None, y), (x, g, None, off)]:
        with pytest.raises(M.MoeError) as ei:
            M.moe_norm_forward(args[0], M.MOE_F32, M.MOE_NORM_RMS, args[1], args[2], 0.0, T, m, args[3])
        assert ei.value.status == M.MOE_ERR_INVALID_ARG


def test_norm_backward_of_no_rows():
    dg, db = torch.full((136,), 3.0, device="cuda"), torch.full((136,), 3.0, device="cuda")
    M.moe_norm_backward(None, None, M.MOE_F32, M.MOE_NORM_LAYER, None, None, None, 0, 128, None, dg[:128], db[:128])
    assert bool((dg[:128] == 0).all()) and bool((db[:128] == 0).all())
    assert bool((dg[128:] == 3).all()) and bool((db[128:] == 3).all())


@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
def test_norm_gradients_against_differences(layer):
    """The kernel's gradients against central differences of the 64-bit
    forward along random directions: with step s the difference is off by
    s^2 / 6 times a third derivative (measured by halving s) and by the
    64-bit rounding 2^-52 |loss| / s."""
    T, m, eps = 6, 200, 1e-5
    rng = np.random.default_rng(0)
    x, gamma, beta, dy = (rng.standard_normal(s).astype(np.float32) for s in ((T, m), (m,), (m,), (T, m)))
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()
    kind = M.MOE_NORM_LAYER if layer else M.MOE_NORM_RMS
    y, mean, rstd = torch.empty(T, m, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    M.moe_norm_forward(cu(x), M.MOE_F32, kind, cu(gamma), cu(beta) if layer else None, eps, T, m, y,
                       mean if layer else None, rstd)
    dx, dg, db = torch.empty(T, m, device="cuda"), torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    n = M.moe_norm_backward_workspace_size(T, m)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    M.moe_norm_backward(cu(dy), cu(x), M.MOE_F32, kind, cu(gamma), mean if layer else None, rstd, T, m, dx, dg,
                        db if layer else None, ws, n)

    def loss(x_, g_, b_):
        return float((norm_ref(x_, g_, b_ if layer else None, eps, layer)[0] * dy).sum())

    at = [a.astype(np.float64) for a in (x, gamma, beta)]
    for i, grad in enumerate((dx, dg, db) if layer else (dx, dg)):
        d = rng.standard_normal(at[i].shape)

        def diff(s):
            hi, lo = list(at), list(at)
            hi[i], lo[i] = at[i] + s * d, at[i] - s * d
            return (loss(*hi) - loss(*lo)) / (2 * s)

        a, b = diff(2e-4), diff(1e-4)
        got = float((n64(grad) * d).sum())
        # the kernel: (m + 20) u of the terms' magnitudes (test_norm_backward's bounds, summed)
        tol = abs(a - b) + 2.0**-52 * 64 * T * m / 1e-4 + (m + 20) * u * 8 * float((np.abs(n64(grad)) * np.abs(d)).sum() + T * m)
        assert abs(got - b) <= tol, (i, got, b, tol)


# ---- rows in expert order -------------------------------------------------------------


def plan(T, k, E, drop, seed):
    """(inv_perm, rows): moe_dispatch's stable order over random choices of k
    distinct experts, without the dropped assignments (their entries lie
    outside [0, rows))."""
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).reshape(-1) if T else np.zeros(0, int)
    keep = rng.random(T * k) >= drop
    order = np.argsort(np.where(keep, idx, E), kind="stable")
    rows = int(keep.sum())
    inv = rng.choice([-1, -2**31, rows, rows + 5, 2**31 - 1], T * k).astype(np.int64)
    inv[order[:rows]] = np.arange(rows)
    return torch.from_numpy(inv.astype(np.int32)).cuda(), rows


ROW_CASES = [(1, 1, 1, 8, 0.0), (1, 2, 8, 64, 0.0), (5, 2, 8, 72, 0.3), (64, 2, 8, 4096, 0.0), (33, 4, 16, 1000, 0.5),
             (7, 3, 3, 2056, 0.0), (3, 64, 64, 520, 0.2), (9, 6, 33, 9000, 0.9), (1025, 2, 8, 136, 0.1),
             (4, 2, 8, 512, 1.0)]
PAIRS = [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)]
ids = lambda p: "_".join("bf16" if d is BF16 else "f32" for d in p)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,m,drop", ROW_CASES)
def test_permute_rows(T, k, E, m, drop, dtype):
    inv, rows = plan(T, k, E, drop, T + m)
    x = rnd((T, m), dtype, m)
    out = Guarded((rows + 3, m), dtype, 5.0)
    M.moe_permute_rows(x, CODE[dtype], inv, T, m, k, rows, out.t)
    i = inv.cpu().numpy()
    got, ref = n64(out.t), np.full((rows + 3, m), 5.0)
    for a in range(T * k):
        if 0 <= i[a] < rows:
            ref[i[a]] = n64(x[a // k])
    assert np.array_equal(got, ref)  # the rows behind the last stay as they were
    out.intact()


@pytest.mark.parametrize("pair", PAIRS, ids=ids)
@pytest.mark.parametrize("weighted", [True, False], ids=["combine", "permute_backward"])
@pytest.mark.parametrize("T,k,E,m,drop", ROW_CASES)
def test_combine_rows(T, k, E, m, drop, weighted, pair):
    rt, ot = pair
    inv, rows = plan(T, k, E, drop, T + m)
    r = rnd((rows, m), rt, m + 1)
    w = rnd((T, k), F32, m + 2)
    there = (inv.view(T, k) >= 0) & (inv.view(T, k) < rows)
    w[~there] = float("nan")  # a dropped assignment's weight is not used
    out = Guarded((T, m), ot)
    if weighted:
        M.moe_combine_rows(r, CODE[rt], inv, w, T, m, k, rows, out.t, CODE[ot])
    else:
        M.moe_permute_rows_backward(r, CODE[rt], inv, T, m, k, rows, out.t, CODE[ot])
    i, w64, r64, ok = inv.cpu().numpy().reshape(T, k), n64(w), n64(r), there.cpu().numpy()
    ref, mag = np.zeros((T, m)), np.zeros((T, m))
    for t in range(T):
        for j in range(k):
            if ok[t, j]:
                term = r64[i[t, j]] * (w64[t, j] if weighted else 1.0)
                ref[t] += term
                mag[t] += np.abs(term)
    check(out.t, ref, k * u * mag + U[ot] * np.abs(ref) * (1 + 2.0**-7) + U[ot] * k * u * mag, "y")
    assert np.all(n64(out.t)[~ok.any(1)] == 0.0)  # tokens without any row
    out.intact()


@pytest.mark.parametrize("pair", PAIRS, ids=ids)
@pytest.mark.parametrize("T,k,E,m,drop", ROW_CASES)
def test_combine_rows_backward(T, k, E, m, drop, pair):
    rt, tt = pair
    inv, rows = plan(T, k, E, drop, T + m)
    r, dy, w = rnd((rows, m), rt, m + 1), rnd((T, m), tt, m + 3), rnd((T, k), F32, m + 2)
    out, dw = Guarded((rows + 2, m), rt, 5.0), Guarded((T, k), F32)
    M.moe_combine_rows_backward(dy, CODE[tt], r, CODE[rt], inv, w, T, m, k, rows, out.t, dw.t)
    i, w64, r64, d64 = inv.cpu().numpy().reshape(T, k), n64(w), n64(r), n64(dy)
    ref, dref, mag = np.full((rows + 2, m), 5.0), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if 0 <= i[t, j] < rows:
                ref[i[t, j]] = w64[t, j] * d64[t]
                dref[t, j] = d64[t] @ r64[i[t, j]]
                mag[t, j] = np.abs(d64[t]) @ np.abs(r64[i[t, j]])
    assert np.all(n64(out.t)[rows:] == 5.0)
    check(out.t, ref, (u + U[rt]) * np.abs(ref) * (1 + 2.0**-7), "dy_perm")
    check(dw.t, dref, m * u * mag, "d_topk_w")
    for o in (out, dw):
        o.intact()
    if rows:  # each output alone
        one, onew = torch.full_like(out.t, 5.0), torch.empty_like(dw.t)
        M.moe_combine_rows_backward(dy, CODE[tt], None, CODE[rt], inv, w, T, m, k, rows, one, None)
        M.moe_combine_rows_backward(dy, CODE[tt], r, CODE[rt], inv, None, T, m, k, rows, None, onew)
        assert torch.equal(one, out.t) and torch.equal(onew, dw.t)


def test_combine_masks_infinities_of_rows_without_an_assignment():
    """Rows that no token names may hold anything."""
    inv = torch.tensor([0, -1, 3, 9, -1, -1], dtype=torch.int32, device="cuda")
    r = rnd((5, 64), F32, 1)
    r[1], r[2], r[4] = float("inf"), float("nan"), -float("inf")
    w = torch.ones(3, 2, device="cuda")
    y = torch.empty(3, 64, device="cuda")
    M.moe_combine_rows(r, M.MOE_F32, inv, w, 3, 64, 2, 5, y, M.MOE_F32)
    assert torch.equal(y, torch.stack([r[0], r[3], torch.zeros(64, device="cuda")]))
    dw = torch.empty(3, 2, device="cuda")
    M.moe_combine_rows_backward(y, M.MOE_F32, r, M.MOE_F32, inv, None, 3, 64, 2, 5, None, dw)
    assert torch.all(torch.isfinite(dw)) and bool((dw[2] == 0).all()) and float(dw[0, 1]) == 0


def test_permute_adjoint():
    """<permute(x), g> = <x, permute_backward(g)> exactly on small integers."""
    T, k, E, m = 37, 3, 8, 200
    inv, rows = plan(T, k, E, 0.2, 9)
    g = torch.Generator().manual_seed(0)
    x = torch.randint(-8, 9, (T, m), generator=g).to(BF16).cuda()
    gr = torch.randint(-8, 9, (rows, m), generator=g).to(BF16).cuda()
    xp, dx = torch.empty(rows, m, dtype=BF16, device="cuda"), torch.empty(T, m, dtype=F32, device="cuda")
    M.moe_permute_rows(x, M.MOE_BF16, inv, T, m, k, rows, xp)
    M.moe_permute_rows_backward(gr, M.MOE_BF16, inv, T, m, k, rows, dx, M.MOE_F32)
    assert float((xp.double() * gr.double()).sum()) == float((x.double() * dx.double()).sum())


def test_combine_gradients_against_differences():
    """The combine is linear in the rows and in the weights, so a central
    difference of the 64-bit forward is exact up to 64-bit rounding."""
    T, k, E, m = 11, 2, 8, 136
    inv, rows = plan(T, k, E, 0.2, 4)
    r, dy, w = rnd((rows, m), F32, 1), rnd((T, m), F32, 2), rnd((T, k), F32, 3)
    dr, dw = torch.zeros(rows, m, device="cuda"), torch.empty(T, k, device="cuda")
    M.moe_combine_rows_backward(dy, M.MOE_F32, r, M.MOE_F32, inv, w, T, m, k, rows, dr, dw)
    i = inv.cpu().numpy().reshape(T, k)

    def loss(r_, w_):
        return sum(w_[t, j] * (r_[i[t, j]] @ n64(dy)[t]) for t in range(T) for j in range(k) if 0 <= i[t, j] < rows)

    rng = np.random.default_rng(1)
    d, e = rng.standard_normal((rows, m)), rng.standard_normal((T, k))
    r64, w64 = n64(r), n64(w)
    s = 0.5
    num = (loss(r64 + s * d, w64) - loss(r64 - s * d, w64)) / (2 * s)
    assert abs(num - (n64(dr) * d).sum()) <= 4 * u * (np.abs(n64(dr)) * np.abs(d)).sum()
    num = (loss(r64, w64 + s * e) - loss(r64, w64 - s * e)) / (2 * s)
    mag = sum(abs(e[t, j]) * (np.abs(r64[i[t, j]]) @ np.abs(n64(dy)[t])) for t in range(T) for j in range(k)
              if 0 <= i[t, j] < rows)
    assert abs(num - (n64(dw) * e).sum()) <= (m + 4) * u * mag


def test_offsets_past_32_bits():
    """Rows whose byte and element offsets pass 2^32 and 2^31."""
    m, T, k = 4096, 280_000, 2
    rows = T * k  # 560,000 x 4096 bf16: 2.29e9 elements, 4.6 GB
    inv = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda")
    x = torch.randint(-99, 100, (T, m), dtype=torch.int8, device="cuda").to(BF16)
    out = torch.empty(rows, m, dtype=BF16, device="cuda")
    M.moe_permute_rows(x, M.MOE_BF16, inv, T, m, k, rows, out)
    pick = torch.tensor([0, 1, 1000, T // 2, T - 2, T - 1], device="cuda")
    for j in range(k):
        assert torch.equal(out[rows - 1 - (pick * k + j)], x[pick])
    w = torch.tensor([[0.5, 0.25]], device="cuda").expand(T, k).contiguous()
    back = torch.empty_like(x)
    M.moe_combine_rows(out, M.MOE_BF16, inv, w, T, m, k, rows, back, M.MOE_BF16)
    assert torch.equal(back, (x.float() * 0.75).to(BF16))
    dw = torch.empty(T, k, device="cuda")
    M.moe_combine_rows_backward(x, M.MOE_BF16, out, M.MOE_BF16, inv, w, T, m, k, rows, out, dw)
    s = x[pick].double().square().sum(1)
    assert torch.equal(dw[pick, 0].double(), dw[pick, 1].double())
    assert torch.all((dw[pick, 0].double() - s).abs() <= m * u * s)
    del out, back
    xx = x.repeat(2, 1)  # 560,000 rows through the norm
    y = torch.empty_like(xx)
    g = torch.ones(m, device="cuda")
    rstd = torch.empty(len(xx), device="cuda")
    M.moe_norm_forward(xx, M.MOE_BF16, M.MOE_NORM_RMS, g, None, 1e-5, len(xx), m, y, None, rstd)
    assert torch.equal(y[T:], y[:T]) and torch.equal(rstd[T:], rstd[:T])
    dx = torch.empty_like(xx)
    M.moe_norm_backward(y, xx, M.MOE_BF16, M.MOE_NORM_RMS, g, None, rstd, len(xx), m, dx, None, None)
    assert torch.equal(dx[T:], dx[:T])


def test_as_many_tokens_as_an_int_counts():
    """T = 2^31 - 8 with k = 1: no loop over tokens may step past the last one
    in 32 bits.  Four tokens have a row; the products are exact."""
    T, m, rows = 2**31 - 8, 8, 4
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("needs 70 GB")
    toks = torch.tensor([0, 2**22, 2**31 - 2**22, T - 1], device="cuda")
    inv = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    inv[toks] = torch.arange(rows, dtype=torch.int32, device="cuda")
    x = torch.full((T, m), 2.0, dtype=BF16, device="cuda")
    x[toks] = torch.tensor([1.0, 3.0, 5.0, 7.0], dtype=BF16, device="cuda")[:, None]
    yp = torch.full((rows, m), 0.5, dtype=BF16, device="cuda")
    w = torch.full((T,), 4.0, dtype=F32, device="cuda")

    xp = torch.zeros((rows, m), dtype=BF16, device="cuda")
    M.moe_permute_rows(x, M.MOE_BF16, inv, T, m, 1, rows, xp)
    assert xp[:, 0].tolist() == [1.0, 3.0, 5.0, 7.0] and bool((xp == xp[:, :1]).all())

    dyp = torch.zeros_like(yp)
    dw = torch.full((T,), 9.0, dtype=F32, device="cuda")
    M.moe_combine_rows_backward(x, M.MOE_BF16, yp, M.MOE_BF16, inv, w, T, m, 1, rows, dyp, dw)
    assert dyp[:, 0].tolist() == [4.0, 12.0, 20.0, 28.0] and bool((dyp == dyp[:, :1]).all())
    assert dw[toks].tolist() == [4.0, 12.0, 20.0, 28.0]
    dw[toks] = 0.0
    assert float(dw.abs().amax()) == 0.0
    del dw

    M.moe_combine_rows(yp, M.MOE_BF16, inv, w, T, m, 1, rows, x, M.MOE_BF16)
    assert bool((x[toks] == 2.0).all())
    x[toks] = 0.0
    assert float(x.amax()) == 0.0 and float(x.amin()) == 0.0
    del x, inv, w
    torch.cuda.empty_cache()


# Calls that move 128 MB or more read their inputs as data not to be kept; the
# same rows in smaller calls must give the same bits, row by row.
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("m", [1000, 4096, 16376])
def test_large_norms_match_small_ones(m, layer, dtype):
    es = 2 if dtype == BF16 else 4
    T = 4 * ((64 << 20) // (4 * m * es) + 1)
    kind = M.MOE_NORM_LAYER if layer else M.MOE_NORM_RMS
    x, dy, gamma = rnd((T, m), dtype, 1, shift=0.25), rnd((T, m), dtype, 2), rnd((m,), F32, 3)
    beta = rnd((m,), F32, 4) if layer else None

    def call(lo, n):
        xs, dys = x[lo:lo + n], dy[lo:lo + n]
        y, dx = torch.empty_like(xs), torch.empty_like(xs)
        mean, rstd = torch.empty(n, device="cuda") if layer else None, torch.empty(n, device="cuda")
        dg, db = torch.empty(m, device="cuda"), torch.empty(m, device="cuda") if layer else None
        M.moe_norm_forward(xs, CODE[dtype], kind, gamma, beta, 1e-5, n, m, y, mean, rstd)
        b = M.moe_norm_backward_workspace_size(n, m)
        ws = torch.empty(max(b, 256), dtype=torch.uint8, device="cuda")
        M.moe_norm_backward(dys, xs, CODE[dtype], kind, gamma, mean, rstd, n, m, dx, dg, db, ws, b)
        return y, dx, rstd, dg, db

    y, dx, rstd, dg, db = call(0, T)
    n = T // 4
    parts = [call(i * n, n) for i in range(4)]
    for whole, at in [(y, 0), (dx, 1), (rstd, 2)]:
        assert torch.equal(whole, torch.cat([p[at] for p in parts]))
    for whole, at in [(dg, 3), (db, 4)]:
        if whole is not None:  # each sum is within T u of its terms' magnitudes: |dy h| <= |dy| |h|, |h| <= sqrt(m)
            s = sum(p[at].double() for p in parts)
            mag = dy.double().abs().sum(0) * (m**0.5 if at == 3 else 1.0)
            assert bool(((whole.double() - s).abs() <= 2 * T * u * mag).all())


@pytest.mark.parametrize("pair", PAIRS, ids=ids)
def test_large_rows_match_small_ones(pair):
    td, rd = pair  # of token rows and of expert rows
    T, k, m = 8192, 2, 4104
    R, n = T * k, T // 4
    g = torch.Generator().manual_seed(5)
    small = [torch.randperm(n * k, generator=g).to(torch.int32).cuda() for _ in range(4)]  # a quarter's tokens, its rows
    inv = torch.cat([p + i * n * k for i, p in enumerate(small)])
    x, yp, w = rnd((T, m), td, 1), rnd((R, m), rd, 2), rnd((T, k), F32, 3)

    def call(t0, T, inv):
        xs, ys, ws, R = x[t0:t0 + T], yp[t0 * k:(t0 + T) * k], w[t0:t0 + T], T * k
        xp, out, back = torch.empty(R, m, dtype=td, device="cuda"), torch.empty_like(xs), torch.empty_like(xs)
        dyp, dw = torch.empty_like(ys), torch.empty_like(ws)
        M.moe_permute_rows(xs, CODE[td], inv, T, m, k, R, xp)
        M.moe_permute_rows_backward(ys, CODE[rd], inv, T, m, k, R, back, CODE[td])
        M.moe_combine_rows(ys, CODE[rd], inv, ws, T, m, k, R, out, CODE[td])
        M.moe_combine_rows_backward(xs, CODE[td], ys, CODE[rd], inv, ws, T, m, k, R, dyp, dw)
        return xp, back, out, dyp, dw

    whole = call(0, T, inv)
    parts = [call(i * n, n, small[i]) for i in range(4)]
    for i, a in enumerate(whole):
        assert torch.equal(a, torch.cat([p[i] for p in parts]))
    assert torch.equal(whole[0][inv.long()], x.repeat_interleave(k, 0))
