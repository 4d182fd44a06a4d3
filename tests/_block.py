"""64-bit definitions of the trainable block's operators, each with the bound that
counts its roundings (torch tensors in float64, on whatever device).

u = 2^-24 is half an fp32 step, U[dtype] half a step of the stored type.  A sum of n
products on the matrix cores is within 2 n u sum|terms| of its exact value: each of its
additions, in any order, is rounded or truncated to fp32 (at most a whole step, 2 u);
values in two parts make twice as many products.  sigmoid(g): exp(-g) carries its argument's rounding, |g| u, and its own steps,
the sum and the division or reciprocal one each: within (2 |g| + 8) u of its value.
"""
import torch

u = 2.0**-24
U = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8}


def hidden_step(rows, E, dtype):
    """Half a step of a hidden row's values: in bf16, two parts for up to 32 rows an expert,
    the second rounded to half a step of what the first leaves (at most 2^-8 of the value)."""
    few = rows and -(-rows // min(rows, E)) <= 32
    return 2.0**-16 if dtype == torch.bfloat16 and few else U[dtype]


TINY = 1e-36  # results and terms below the normal range round absolutely


def ranges(offsets, rows, E):
    """The row ranges as the operators read them: clamped, none decreasing."""
    if offsets is None:
        return [(0, rows)]
    o = [min(max(int(v), 0), rows) for v in offsets.tolist()]
    out, at = [], 0
    for e in range(E):
        at = max(at, o[e])
        end = max(at, o[e + 1])
        out.append((at, end))
    return out


def _mm(a, b):
    """a b and the sum of its terms' magnitudes."""
    return a @ b, a.abs() @ b.abs()


def forward(x, wg, wu, wd, offsets, perm, topk, rows, dtype):
    """(y, gate, up) and their bounds; rows of no range are NaN in the results."""
    E, m, p = wg.shape
    y = torch.full((rows, m), float("nan"), dtype=torch.float64, device=x.device)
    g, up = (torch.full((rows, p), float("nan"), dtype=torch.float64, device=x.device) for _ in range(2))
    by, bg, bu = torch.zeros_like(y), torch.zeros_like(g), torch.zeros_like(up)
    r_, h_ = U[dtype], hidden_step(rows, E, dtype)
    for e, (lo, hi) in enumerate(ranges(offsets, rows, E)):
        if lo == hi:
            continue
        t = torch.arange(lo, hi, device=x.device)
        if perm is not None:
            t = (perm[lo:hi].long() // topk).clamp(0, len(x) - 1)
        xe, W = x[t].double(), [w[e].double() for w in (wg, wu, wd)]
        ge, ga = _mm(xe, W[0])
        ue, ua = _mm(xe, W[1])
        eg, eu = 2 * (m + 1) * u * ga, 2 * (m + 1) * u * ua
        s = torch.sigmoid(ge)
        h = ge * s * ue
        # silu' lies in (-0.1, 1.1); the sigmoid's error and two products
        eh = 1.1 * eg * (ue.abs() + eu) + (ge * s).abs() * eu + h.abs() * (2 * ge.abs() + 12) * u + h_ * h.abs()
        ye, ya = _mm(h, W[2])
        y[lo:hi], g[lo:hi], up[lo:hi] = ye, ge, ue
        by[lo:hi] = eh @ W[2].abs() + 2 * (2 * p + 1) * u * ya + r_ * ye.abs()
        bg[lo:hi], bu[lo:hi] = eg + r_ * ge.abs(), eu + r_ * ue.abs()
    return (y, g, up), (by, bg, bu)


def backward(dy, x, wg, wu, wd, gate, up, offsets, perm, topk, rows, dtype):
    """(dx, dwg, dwu, dwd) and their bounds."""
    E, m, p = wg.shape
    dx = torch.full((rows, m), float("nan"), dtype=torch.float64, device=x.device)
    out = [dx] + [torch.zeros(w.shape, dtype=torch.float64, device=x.device) for w in (wg, wu, wd)]
    bnd = [torch.zeros_like(o) for o in out]
    r_, h_ = U[dtype], hidden_step(rows, E, dtype)
    for e, (lo, hi) in enumerate(ranges(offsets, rows, E)):
        if lo == hi:
            continue
        n = hi - lo
        t = torch.arange(lo, hi, device=x.device)
        if perm is not None:
            t = (perm[lo:hi].long() // topk).clamp(0, len(x) - 1)
        xe, d, g, q = x[t].double(), dy[lo:hi].double(), gate[lo:hi].double(), up[lo:hi].double()
        W = [w[e].double() for w in (wg, wu, wd)]
        dh, da = _mm(d, W[2].T)
        edh = 2 * (m + 1) * u * da
        s = torch.sigmoid(g)
        gs = g * s
        a = q.abs() * (s + gs.abs() * (1 - s))  # bounds the factor of dg and its terms
        dg, du, h = dh * q * (s + gs * (1 - s)), dh * gs, gs * q
        near = (2 * g.abs() + 16) * u
        edg = a * edh + (dh.abs() + edh) * a * near + h_ * dg.abs() * (1 + h_)
        edu = gs.abs() * edh + (dh.abs() + edh) * gs.abs() * near + h_ * du.abs() * (1 + h_)
        eh = h.abs() * near + h_ * h.abs()
        x1, a1 = _mm(dg, W[0].T)
        x2, a2 = _mm(du, W[1].T)
        out[0][lo:hi] = x1 + x2
        bnd[0][lo:hi] = edg @ W[0].abs().T + edu @ W[1].abs().T + 2 * (4 * p + 1) * u * (a1 + a2) + r_ * (x1 + x2).abs()
        for i, (l, v, el, ev) in enumerate([(xe, dg, None, edg), (xe, du, None, edu), (h, d, eh, None)]):
            o, mag = _mm(l.T, v)
            b = 2 * (2 * n + 1) * u * mag + r_ * o.abs()
            b += l.abs().T @ ev if ev is not None else el.T @ v.abs()
            out[i + 1][e], bnd[i + 1][e] = o, b
    return out, bnd


def route_backward(dw, idx, w, dl_add, x, wr, dx_add, E, dtype):
    """(dl, dx, dwr, db) and their bounds."""
    T, k = w.shape
    dw, w, x, wr = dw.double(), w.double(), x.double(), wr.double()
    dot = (w * dw).sum(1, keepdim=True)
    mag = (w * dw).abs().sum(1, keepdim=True)
    v = w * (dw - dot)
    ev = w.abs() * ((k + 1) * u * mag + 3 * u * (dw.abs() + mag))
    hit = idx[:, :, None].long() == torch.arange(E, device=x.device)
    dl, edl, sized = ((hit * q[:, :, None]).sum(1) for q in (v, ev, v.abs()))
    if dl_add is not None:
        dl, sized = dl + dl_add.double(), sized + dl_add.double().abs()
    edl = edl + (k + 1) * u * sized
    dx, mx = _mm(dl, wr.T)
    bx = edl @ wr.T.abs() + 2 * (E + 1) * u * mx
    if dx_add is not None:
        dx, mx = dx + dx_add.double(), mx + dx_add.double().abs()
    bx = bx + 2 * u * mx + U[dtype] * dx.abs()
    dwr, mw = _mm(x.T, dl)
    bw = x.T.abs() @ edl + 2 * (T + 1) * u * mw
    db, bb = dl.sum(0), edl.sum(0) + 2 * (T + 1) * u * dl.abs().sum(0)
    return (dl, dx, dwr, db), (edl + u * dl.abs(), bx, bw, bb)


def check(got, want, bound, what, log=print):
    """Every element within its bound; NaN in `want` is an element that has none."""
    got, bound = got.double(), bound * (1 + 2.0**-6) + TINY  # second-order terms
    there = ~torch.isnan(want)
    assert got.shape == want.shape, what
    err = (got - want).abs()[there]
    assert bool(torch.isfinite(got[there]).all()), f"{what}: not finite"
    worst = float((err / bound[there]).max()) if err.numel() else 0.0
    log(f"  {what}: max|err| {float(err.max()) if err.numel() else 0:.3e}, {worst:.3f} of the bound")
    assert worst <= 1.0, f"{what}: {worst} of the bound"
