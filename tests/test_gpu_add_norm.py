"""The residual norm (moe_add_norm_forward, _backward) against 64-bit definitions.
The bounds count roundings, as in test_gpu_rows.py: u is half an fp32 step, a sum of n
terms is within (n - 1) u sum|terms|, and each other operation adds u of its result."""
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
TINY = 1e-37
EPS = 1e-5


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
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    worst = float(np.max(np.abs(got - ref) / (bar + TINY))) if got.size else 0.0
    log(f"  {what}: {worst:.3f} of the bound")
    assert worst <= 1.0, what


class Guarded:
    def __init__(self, shape, dtype, fill=5):
        n = int(np.prod(shape))
        self.buf = torch.full((n + 256,), 7, dtype=dtype, device="cuda")
        self.t = self.buf[128:128 + n].view(shape)
        self.t.fill_(fill)

    def intact(self):
        assert bool((self.buf[:128] == 7).all()) and bool((self.buf[128 + self.t.numel():] == 7).all())


def reference(x, r, gamma, beta, layer, dtype):
    """s, mean, rstd, y in 64 bits with their bounds (y's before its rounding)."""
    m = x.shape[1]
    s = x + r if r is not None else x
    e_s = u * np.abs(s) if r is not None else 0 * s
    avg = np.abs(s).mean(1)
    mu = s.mean(1) if layer else np.zeros(len(s))
    e_mu = (m + 3) * u * avg if layer else np.zeros(len(s))
    d = s - mu[:, None]
    rs = 1.0 / np.sqrt((d * d).mean(1) + EPS)
    h = d * rs[:, None]
    # the deviations' errors: e_s and e_mu each, and a rounding; they move the mean
    # of squares by at most 2 avg|d e| + e^2
    e_d = e_s + e_mu[:, None] + u * np.abs(d)
    moved = (2 * np.abs(d) * e_d + e_d * e_d).mean(1) * rs * rs
    e_r = 0.5 * ((m + 4) * u + moved) + 4 * u
    y = h * gamma + (beta if beta is not None else 0.0)
    e_h = e_d * rs[:, None] + np.abs(h) * (e_r[:, None] + 3 * u)
    e_y = np.abs(gamma) * e_h + 2 * u * np.abs(h * gamma) + 2 * u * np.abs(y)
    return s, mu, rs, y, e_s, e_mu, rs * e_r, e_y * (1 + 2.0**-7)


SHAPES = [(1, 8), (3, 64), (5, 72), (1, 520), (7, 1000), (4, 2048), (3, 2056), (2, 4096), (6, 5000), (2, 8200), (3, 16384),
          (1100, 64), (2100, 2048), (700, 4104)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("norm", ["layer", "layer_nobeta", "rms"])
@pytest.mark.parametrize("T,m", SHAPES)
def test_forward(T, m, norm, dtype):
    layer = norm != "rms"
    log(f"add norm {norm} {dtype} T={T} m={m}")
    x, r = rnd((T, m), dtype, T * m, 1.0, 0.5), rnd((T, m), dtype, T * m + 1, 2.0, 1.0)
    gamma, beta = rnd((m,), F32, 1, 0.2, 1.0), rnd((m,), F32, 2, 0.3) if norm == "layer" else None
    outs = dict(sum=Guarded((T, m), dtype), y=Guarded((T, m), dtype), codes=Guarded((T, m), torch.int8),
                scale=Guarded((T,), F32), mean=Guarded((T,), F32), rstd=Guarded((T,), F32))
    kind = M.MOE_NORM_LAYER if layer else M.MOE_NORM_RMS
    o = {n: g.t for n, g in outs.items()}
    if not layer:
        o["mean"] = None
    M.moe_add_norm_forward(x, r, CODE[dtype], kind, gamma, beta, EPS, T, m, **o)
    torch.cuda.synchronize()
    s, mu, rs, y, e_s, e_mu, e_r, e_y = reference(n64(x), n64(r), n64(gamma), n64(beta), layer, dtype)
    check(o["sum"], s, e_s + U[dtype] * np.abs(s) * (1 + u), "sum")
    check(o["rstd"], rs, e_r, "rstd")
    if layer:
        check(o["mean"], mu, e_mu, "mean")
    check(o["y"], y, e_y + U[dtype] * np.abs(y) * (1 + 2.0**-7), "y")
    # the scale: a power of two, the smallest that 127 steps of reach the row (as far as y's error lets that be seen)
    scale, codes = n64(o["scale"]), n64(o["codes"])
    top, slack = np.abs(y).max(1), e_y.max(1)
    assert np.all(np.log2(scale) % 1 == 0)
    assert np.all(top - slack <= 127 * scale) and np.all(top + slack > 127 * scale / 2)
    assert np.abs(codes).max() <= 127
    check(o["codes"].float() * o["scale"][:, None], y, 0.5 * scale[:, None] + e_y, "codes")
    for g in outs.values():
        g.intact()
    # each output alone: the same bits
    for part in (("y",), ("codes", "scale"), ("sum", "y")):
        alone = {n: torch.empty_like(o[n]) if n in part else None for n in ("sum", "y", "codes", "scale")}
        M.moe_add_norm_forward(x, r, CODE[dtype], kind, gamma, beta, EPS, T, m, **alone)
        assert all(torch.equal(alone[n], o[n]) for n in part), part


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("T,m", SHAPES)
def test_backward(T, m, norm, dtype):
    layer = norm == "layer"
    log(f"add norm gradient {norm} {dtype} T={T} m={m}")
    s, dy, ds = rnd((T, m), dtype, 3, 2.0, 0.5), rnd((T, m), dtype, 4), rnd((T, m), dtype, 5, 1.5)
    gamma = rnd((m,), F32, 6, 0.2, 1.0)
    x64 = n64(s)
    mu = x64.mean(1) if layer else np.zeros(T)
    mean = torch.from_numpy(mu).float().cuda() if layer else None
    rstd = torch.from_numpy(1 / np.sqrt(((x64 - mu[:, None])**2).mean(1) + EPS)).float().cuda()
    n = M.moe_norm_backward_workspace_size(T, m)
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")
    kind = M.MOE_NORM_LAYER if layer else M.MOE_NORM_RMS
    dx, dg, db = Guarded((T, m), dtype), Guarded((m,), F32), Guarded((m,), F32)
    M.moe_add_norm_backward(dy, ds, s, CODE[dtype], kind, gamma, mean, rstd, T, m, dx.t, dg.t, db.t if layer else None, ws, n)
    torch.cuda.synchronize()
    r, g, d = n64(rstd)[:, None], n64(gamma), n64(dy)
    mu = n64(mean)[:, None] if layer else 0.0
    h, w = (x64 - mu) * r, d * g
    a, b = (w * h).mean(1, keepdims=True), w.mean(1, keepdims=True) if layer else 0.0
    aa, ab = np.abs(w * h).mean(1, keepdims=True), np.abs(w).mean(1, keepdims=True) if layer else 0.0
    part = r * (w - h * a - b)
    want = n64(ds) + part
    # u of each product and difference on |w|, |h a| and |b|; the averages' m + 3 roundings
    e = r * (8 * u * (np.abs(w) + np.abs(h) * np.abs(a) + np.abs(b)) + (m + 6) * u * (np.abs(h) * aa + ab))
    check(dx.t, want, e + u * np.abs(part) + 2 * u * np.abs(want) + U[dtype] * np.abs(want) * (1 + 2.0**-7), "dx")
    check(dg.t, (d * h).sum(0), (T + 6) * u * np.abs(d * h).sum(0), "dgamma")
    if layer:
        check(db.t, d.sum(0), (T + 3) * u * np.abs(d).sum(0), "dbeta")
    for o in (dx, dg, db):
        o.intact()
    # without dsum: the norm's own gradient, within the same bound less dsum's addition (not
    # moe_norm_backward's bits: the compiler fuses products and sums in each form as it likes);
    # over dy or dsum the same bits
    plain = torch.empty_like(dx.t)
    M.moe_add_norm_backward(dy, None, s, CODE[dtype], kind, gamma, mean, rstd, T, m, plain, None, None)
    check(plain, part, e + u * np.abs(part) + U[dtype] * np.abs(part) * (1 + 2.0**-7), "dx without dsum")
    for where in (0, 1):
        v = [dy.clone(), ds.clone()]
        M.moe_add_norm_backward(v[0], v[1], s, CODE[dtype], kind, gamma, mean, rstd, T, m, v[where], None, None)
        assert torch.equal(v[where], dx.t)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,m", [(1, 64), (900, 264), (333, 4096), (40, 9000)])
def test_in_place_and_without_residual(T, m, dtype):
    """sum over the residual, y over x; and without a residual the norm's own rows."""
    x, r, gamma = rnd((T, m), dtype, 1), rnd((T, m), dtype, 2, 3.0), rnd((m,), F32, 3, 0.2, 1.0)
    s, y = torch.empty_like(x), torch.empty_like(x)
    M.moe_add_norm_forward(x, r, CODE[dtype], M.MOE_NORM_RMS, gamma, None, EPS, T, m, s, y)
    for a, b in (("r", "x"), ("x", "r")):
        v = {"x": x.clone(), "r": r.clone()}
        M.moe_add_norm_forward(v["x"], v["r"], CODE[dtype], M.MOE_NORM_RMS, gamma, None, EPS, T, m, v[a], v[b])
        assert torch.equal(v[a], s) and torch.equal(v[b], y)
    M.moe_add_norm_forward(x, None, CODE[dtype], M.MOE_NORM_RMS, gamma, None, EPS, T, m, s, y)
    _, _, _, want, _, _, _, e_y = reference(n64(x), None, n64(gamma), None, False, dtype)
    assert torch.equal(s, x)
    check(y, want, e_y + U[dtype] * np.abs(want) * (1 + 2.0**-7), "y without residual")


def test_special_rows():
    """Zero rows give scale 1 and zero codes; a non-finite row stays alone; ties round to even."""
    m = 256
    x, r = rnd((6, m), F32, 1), rnd((6, m), F32, 2)
    gamma = torch.ones(m, device="cuda")
    s, y, scale = torch.empty_like(x), torch.empty_like(x), torch.empty(6, device="cuda")
    codes = torch.empty(6, m, dtype=torch.int8, device="cuda")
    M.moe_add_norm_forward(x, r, M.MOE_F32, M.MOE_NORM_RMS, gamma, None, EPS, 6, m, s, y, codes, scale)
    x2, r2 = x.clone(), r.clone()
    x2[1], r2[1] = 1.5, -1.5
    x2[3, 7] = float("nan")
    r2[4, 200] = float("inf")
    out = [torch.empty_like(t) for t in (s, y, codes, scale)]
    M.moe_add_norm_forward(x2, r2, M.MOE_F32, M.MOE_NORM_RMS, gamma, None, EPS, 6, m, *out)
    for a, b in zip(out, (s, y, codes, scale)):
        assert torch.equal(a[[0, 2, 5]], b[[0, 2, 5]])
    assert float(out[3][1]) == 1.0 and not bool(out[2][1].any()) and not bool(out[1][1].any())
    # eps = 0 and a row of +-1 and halves that the norm leaves as they are: rms 1 -> y = x, steps of 2^-6
    t = torch.zeros(1, 64, device="cuda")
    t[0, :32] = 1.0
    t[0, 32:] = -1.0
    out = [torch.empty(1, 64, device="cuda"), torch.empty(1, 64, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")]
    gamma = torch.full((64,), 1.0, device="cuda")
    gamma[0], gamma[1], gamma[33] = 2.5 / 64, 3.5 / 64, 0.5 / 64  # ties: 2.5 -> 2, 3.5 -> 4, -0.5 -> 0
    M.moe_add_norm_forward(t, None, M.MOE_F32, M.MOE_NORM_RMS, gamma, None, 0.0, 1, 64, None, *out)
    assert float(out[2]) == 2.0**-6 and out[1][0, [0, 1, 2, 32, 33]].tolist() == [2, 4, 64, -64, 0]


def test_graph_and_stream():
    T, m = 300, 1032
    x, r, gamma = rnd((T, m), BF16, 1), rnd((T, m), BF16, 2), rnd((m,), F32, 3, 0.2, 1.0)
    dy, ds = rnd((T, m), BF16, 4), rnd((T, m), BF16, 5)
    n = M.moe_norm_backward_workspace_size(T, m)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    new = lambda: [torch.empty_like(x), torch.empty_like(x), torch.empty(T, m, dtype=torch.int8, device="cuda"),  # noqa: E731
                   torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(x), torch.empty(m, device="cuda")]

    def step(o):
        M.moe_add_norm_forward(x, r, M.MOE_BF16, M.MOE_NORM_RMS, gamma, None, EPS, T, m, o[0], o[1], o[2], o[3], None, o[4])
        M.moe_add_norm_backward(dy, ds, o[0], M.MOE_BF16, M.MOE_NORM_RMS, gamma, None, o[4], T, m, o[5], o[6], None, ws, n)

    a, b = new(), new()
    step(a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(b)
    for _ in range(3):
        for t in b:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        x.mul_(1.5)
        step(a)
        torch.cuda.synchronize()


def test_codes_feed_the_int8_product():
    """The codes and scales as moe_matmul_i8 takes them: its rows equal the product of the values they stand for."""
    T, m, N = 40, 512, 264
    x, r, gamma = rnd((T, m), BF16, 1), rnd((T, m), BF16, 2), rnd((m,), F32, 3, 0.2, 1.0)
    codes, scale = torch.empty(T, m, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    M.moe_add_norm_forward(x, r, M.MOE_BF16, M.MOE_NORM_RMS, gamma, None, EPS, T, m, None, None, codes, scale)
    g = torch.Generator().manual_seed(7)
    w = torch.randint(-127, 128, (1, N, m), generator=g, dtype=torch.int8).cuda()
    sw = torch.full((1, N), 2.0**-9, device="cuda")
    y = torch.empty(T, N, device="cuda")
    M.moe_matmul_i8(codes, scale, w, sw, None, None, T, 1, T, m, N, 1, y, M.MOE_F32)
    want = (codes.double() * scale.double()[:, None]) @ (w[0].double() * 2.0**-9).T
    # the integer sum is below 2^24 and both scales are powers of two: the product is exact
    assert torch.equal(y.double(), want)
