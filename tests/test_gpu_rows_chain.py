"""The row operators run together, as a layer's caller uses them: a training
step through norm, dispatch, linear experts and combine with its backward
pass, an int8 serving step, and both captured into a HIP graph, on other
streams and two at a time."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

from _gpu import log

pytestmark = pytest.mark.gpu

u = 2.0**-24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


def rnd(shape, seed, scale=1.0, shift=0.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).cuda()


class Layer:
    """A norm, a router, linear experts We [E][m][m] and a combine: buffers and one training step."""

    def __init__(self, T, m, E, k, layer, seed):
        self.T, self.m, self.E, self.k, self.layer = T, m, E, k, layer
        self.kind = M.MOE_NORM_LAYER if layer else M.MOE_NORM_RMS
        self.x, self.dy = rnd((T, m), seed, 1.5, 0.4), rnd((T, m), seed + 1)
        self.gamma, self.beta = rnd((m,), seed + 2, 0.2, 1.0), rnd((m,), seed + 3, 0.1) if layer else None
        self.wg, self.we = rnd((m, E), seed + 4, 0.05), rnd((E, m, m), seed + 5, m**-0.5)
        f = lambda *s: torch.empty(*s, device="cuda")
        i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
        R = T * k
        self.xn, self.rstd, self.mean = f(T, m), f(T), f(T) if layer else None
        self.idx, self.w, self.counts, self.offsets, self.perm, self.inv = i(T, k), f(T, k), i(E), i(E + 1), i(R), i(R)
        self.xp, self.yp, self.y = f(R, m), f(R, m), f(T, m)
        self.dyp, self.dw, self.dxp, self.dxn = f(R, m), f(T, k), f(R, m), f(T, m)
        self.dx, self.dg, self.db = f(T, m), f(m), f(m) if layer else None
        self.n = M.moe_norm_backward_workspace_size(T, m)
        self.ws = torch.empty(self.n, dtype=torch.uint8, device="cuda")

    def route(self):
        T, m, E, k = self.T, self.m, self.E, self.k
        M.moe_norm_forward(self.x, M.MOE_F32, self.kind, self.gamma, self.beta, 1e-5, T, m, self.xn, self.mean, self.rstd)
        M.moe_route_topk(self.xn, M.MOE_F32, self.wg, None, T, m, E, k, 0, None, self.idx, self.w)
        M.moe_dispatch(self.idx, T, E, k, self.counts, self.offsets, self.perm, self.inv)

    def forward(self):
        M.moe_permute_rows(self.xn, M.MOE_F32, self.inv, self.T, self.m, self.k, self.T * self.k, self.xp)

    def combine(self):
        M.moe_combine_rows(self.yp, M.MOE_F32, self.inv, self.w, self.T, self.m, self.k, self.T * self.k, self.y, M.MOE_F32)

    def combine_backward(self):
        M.moe_combine_rows_backward(self.dy, M.MOE_F32, self.yp, M.MOE_F32, self.inv, self.w, self.T, self.m, self.k,
                                    self.T * self.k, self.dyp, self.dw)

    def backward(self):
        M.moe_permute_rows_backward(self.dxp, M.MOE_F32, self.inv, self.T, self.m, self.k, self.T * self.k, self.dxn,
                                    M.MOE_F32)
        M.moe_norm_backward(self.dxn, self.x, M.MOE_F32, self.kind, self.gamma, self.mean, self.rstd, self.T, self.m,
                            self.dx, self.dg, self.db, self.ws, self.n)

    def experts(self, src, dst, transposed):
        o = self.offsets.tolist()
        for e in range(self.E):
            if o[e + 1] > o[e]:
                torch.mm(src[o[e]:o[e + 1]], self.we[e].t().contiguous() if transposed else self.we[e], out=dst[o[e]:o[e + 1]])

    def step(self):
        self.route()
        self.forward()
        self.experts(self.xp, self.yp, False)
        self.combine()
        self.combine_backward()
        self.experts(self.dyp, self.dxp, True)
        self.backward()


@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("T,m,E,k", [(1, 64, 8, 2), (40, 192, 8, 2), (300, 128, 12, 3)])
def test_training_step(T, m, E, k, layer):
    """Against the chain's 64-bit gradients for the routing the GPU took.  Every
    stage is a sum of at most m terms or k terms with a few more roundings;
    the bounds run the same chain on magnitudes."""
    L = Layer(T, m, E, k, layer, T + m)
    L.step()
    torch.cuda.synchronize()
    d = lambda t: t.double().cpu()
    x, gamma = d(L.x).requires_grad_(), d(L.gamma).requires_grad_()
    beta = d(L.beta).requires_grad_() if layer else None
    w, idx = d(L.w).requires_grad_(), L.idx.long().cpu()
    mu = x.mean(1, keepdim=True) if layer else torch.zeros(T, 1, dtype=torch.float64)
    r = ((x - mu).square().mean(1, keepdim=True) + 1e-5).rsqrt()
    h = (x - mu) * r
    xn = h * gamma + (beta if layer else 0.0)
    xn.retain_grad()
    we = d(L.we)
    rows = torch.stack([torch.stack([xn[t] @ we[idx[t, j]] for j in range(k)]) for t in range(T)])
    y = (w[:, :, None] * rows).sum(1)
    (y * d(L.dy)).sum().backward()
    with torch.no_grad():
        a = lambda t: t.detach().abs()
        avg = a(x).mean(1, keepdim=True)
        e_xn = u * ((2 * m + 40) * (avg * r + a(h)) * a(gamma) + 4 * a(xn))  # the norm's own error
        mag = torch.stack([torch.stack([(a(xn)[t] + e_xn[t] / (u * m)) @ a(we[idx[t, j]]) for j in range(k)]) for t in range(T)])
        bar_y = (m + k + 8) * u * (a(w)[:, :, None] * mag).sum(1)
        bar_w = (2 * m + 8) * u * (mag * a(d(L.dy))[:, None, :]).sum(2)
        dmag = torch.stack([sum(a(w)[t, j] * (a(d(L.dy))[t] @ a(we[idx[t, j]]).t()) for j in range(k)) for t in range(T)])
        v = dmag * a(gamma)
        noise = 1 + (avg * r)  # h is off by the mean's error too
        bar_x = (4 * m + 80) * u * r * (v + (a(h) + noise) * (v * (a(h) + noise)).mean(1, keepdim=True) + v.mean(1, keepdim=True))
        bar_g = (4 * m + T + 60) * u * (dmag * (a(h) + noise)).sum(0)
        bar_b = (m + T + 20) * u * dmag.sum(0)
    for got, ref, bar, what in [(L.y, y, bar_y, "y"), (L.dw, w.grad, bar_w, "dw"), (L.dx, x.grad, bar_x, "dx"),
                                (L.dg, gamma.grad, bar_g, "dgamma")] + ([(L.db, beta.grad, bar_b, "dbeta")] if layer else []):
        worst = float(((d(got) - ref.detach()).abs() / (bar + 1e-37)).max())
        log(f"  {what}: {worst:.4f} of the bound")
        assert worst <= 1.0, what


class Int8Step:
    """norm -> route -> dispatch -> codes -> experts' product -> combine."""

    def __init__(self, T, m, p, E, k, seed):
        self.T, self.m, self.p, self.E, self.k = T, m, p, E, k
        bf = torch.bfloat16
        self.x, self.gamma, self.wg = rnd((T, m), seed, dtype=bf), rnd((m,), seed + 1, 0.2, 1.0), rnd((m, E), seed + 2, 0.05)
        g = torch.Generator().manual_seed(seed)
        self.w8 = torch.randint(-127, 128, (E, p, m), generator=g, dtype=torch.int8).cuda()
        self.sw = (torch.rand(E, p, generator=g) * 0.001 + 1e-4).cuda()
        f, i = (lambda *s: torch.empty(*s, device="cuda")), (lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda"))
        R = T * k
        self.xn, self.idx, self.w = torch.empty(T, m, dtype=bf, device="cuda"), i(T, k), f(T, k)
        self.counts, self.offsets, self.perm, self.inv = i(E), i(E + 1), i(R), i(R)
        self.codes, self.sx = torch.empty(T, m, dtype=torch.int8, device="cuda"), f(T)
        self.xp, self.codes_p, self.sx_p = torch.empty(R, m, dtype=bf, device="cuda"), torch.empty(R, m, dtype=torch.int8, device="cuda"), f(R)
        self.yp, self.y = torch.empty(R, p, dtype=bf, device="cuda"), torch.empty(T, p, dtype=bf, device="cuda")

    def step(self, stream=None):
        T, m, p, E, k, s = self.T, self.m, self.p, self.E, self.k, stream
        M.moe_norm_forward(self.x, M.MOE_BF16, M.MOE_NORM_RMS, self.gamma, None, 1e-6, T, m, self.xn, stream=s)
        M.moe_route_topk(self.xn, M.MOE_BF16, self.wg, None, T, m, E, k, 0, None, self.idx, self.w, stream=s)
        M.moe_dispatch(self.idx, T, E, k, self.counts, self.offsets, self.perm, self.inv, stream=s)
        M.moe_quantize_codes_i8(self.xn, T, m, self.codes, self.sx, stream=s)
        M.moe_matmul_i8(self.codes, self.sx, self.w8, self.sw, self.offsets, self.perm, T, k, T * k, m, p, E, self.yp,
                        M.MOE_BF16, stream=s)
        M.moe_combine_rows(self.yp, M.MOE_BF16, self.inv, self.w, T, p, k, T * k, self.y, M.MOE_BF16, stream=s)


@pytest.mark.parametrize("T,m,p,E,k", [(1, 64, 128, 4, 2), (16, 512, 1024, 8, 2), (700, 256, 640, 8, 2), (3000, 512, 768, 4, 2)])
def test_int8_step(T, m, p, E, k):
    L = Int8Step(T, m, p, E, k, T)
    L.step()
    R = T * k
    # rows sorted first, then quantised: the same product bit for bit
    M.moe_permute_rows(L.xn, M.MOE_BF16, L.inv, T, m, k, R, L.xp)
    M.moe_quantize_codes_i8(L.xp, R, m, L.codes_p, L.sx_p)
    yp = torch.empty_like(L.yp)
    M.moe_matmul_i8(L.codes_p, L.sx_p, L.w8, L.sw, L.offsets, None, R, 1, R, m, p, E, yp, M.MOE_BF16)
    assert torch.equal(yp, L.yp)
    # the layer in 64 bits from the codes
    xq = L.codes.double() * L.sx.double()[:, None]
    ref, mag = torch.zeros(T, p, dtype=torch.float64, device="cuda"), torch.zeros(T, p, dtype=torch.float64, device="cuda")
    idx = L.idx.long()
    for e in range(E):
        wv = (L.w8[e].double() * L.sw[e].double()[:, None]).t().contiguous()
        for j in range(k):
            at = (idx[:, j] == e).nonzero().flatten()
            term = (xq[at] @ wv) * L.w[at, j].double()[:, None]
            ref[at] += term
            mag[at] += term.abs()
    # rows rounded to bf16 (2^-8 each), then the fp32 sum and its own rounding
    bar = mag * (2.0**-8 + (k + 4) * u) * (1 + 2.0**-7) + ref.abs() * 2.0**-8 * (1 + 2.0**-6)
    assert bool(((L.y.double() - ref).abs() <= bar + 1e-37).all())


def _outputs(L):
    torch.cuda.synchronize()
    names = [n for n in ("y", "dw", "dx", "dg", "db", "yp", "xn", "dxn") if torch.is_tensor(getattr(L, n, None))]
    return {n: getattr(L, n).clone() for n in names}


def _same(a, b):
    return all(torch.equal(a[n], b[n]) for n in a)


def test_int8_step_captured_and_replayed():
    L = Int8Step(48, 256, 384, 8, 2, 3)
    L.step()
    first = _outputs(L)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        L.step()
    x0 = L.x.clone()
    other = Int8Step(48, 256, 384, 8, 2, 4)
    for turn in range(4):
        for n in ("y", "yp", "xn"):
            getattr(L, n).fill_(float("nan"))
        g.replay()
        other.step()  # the program's own work between replays
        assert _same(_outputs(L), first), turn
    L.x.copy_(x0 * 0.5 + 1)
    g.replay()
    torch.cuda.synchronize()
    replayed = _outputs(L)
    L.step()
    assert _same(_outputs(L), replayed) and not _same(replayed, first)


def test_backward_captured_and_replayed():
    """The whole training step but its dense products in one graph, replayed
    with eager steps on the same buffers between."""
    L = Layer(70, 256, 8, 2, True, 11)
    L.step()
    first = _outputs(L)

    def part():
        L.combine()
        L.combine_backward()
        L.backward()

    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        part()
    for turn in range(4):
        for n in ("y", "dw", "dx", "dg", "db", "dxn"):
            getattr(L, n).fill_(float("nan"))
        L.ws.fill_(0xFF)
        g.replay()
        assert _same(_outputs(L), first), turn
        L.step()
        assert _same(_outputs(L), first), turn


def test_two_streams_at_once():
    """Two training steps and two int8 steps in flight on two streams, each with its own buffers, give the bits each gives alone."""
    A, B = Layer(500, 512, 8, 2, True, 21), Layer(333, 768, 8, 2, False, 22)
    C, D = Int8Step(600, 512, 1024, 8, 2, 23), Int8Step(33, 1024, 512, 8, 2, 24)
    alone = []
    for L in (A, B, C, D):
        L.step()
        alone.append(_outputs(L))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for turn in range(3):
        for L in (A, B, C, D):
            for n in _outputs(L):
                getattr(L, n).fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            A.route(), A.forward(), A.experts(A.xp, A.yp, False)
        with torch.cuda.stream(s2):
            B.route(), B.forward(), B.experts(B.xp, B.yp, False)
        for _ in range(2):
            with torch.cuda.stream(s1):
                A.combine(), A.combine_backward(), C.step()
            with torch.cuda.stream(s2):
                B.combine(), B.combine_backward(), D.step()
        torch.cuda.synchronize()
        A.experts(A.dyp, A.dxp, True), B.experts(B.dyp, B.dxp, True)
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(s1):
                A.backward()
            with torch.cuda.stream(s2):
                B.backward()
        for L, ref in zip((A, B, C, D), alone):
            assert _same(_outputs(L), ref), turn


def test_explicit_stream():
    L = Int8Step(20, 256, 384, 8, 2, 5)
    L.step()
    ref = _outputs(L)
    s = torch.cuda.Stream()
    L.y.fill_(float("nan"))
    torch.cuda.synchronize()
    L.step(stream=s)
    assert _same(_outputs(L), ref)


def test_binding_refuses_small_and_strided_tensors():
    x, g = rnd((8, 64), 0), rnd((64,), 1)
    for bad in [(x[:4], g, x.clone()), (x, g[:32], x.clone()), (x, g, x.clone()[:, :32]), (x, g, x.t().contiguous().t()),
                (x.cpu(), g, x.clone())]:
        with pytest.raises(M.MoeError) as ei:
            M.moe_norm_forward(bad[0], M.MOE_F32, M.MOE_NORM_RMS, bad[1], None, 1e-5, 8, 64, bad[2])
        assert ei.value.status == M.MOE_ERR_INVALID_ARG


def test_binding_refuses_64_bit_indices():
    """torch's own index type, whose halves would be read as int32."""
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.full((4, 2), 0.5, device="cuda")
    inv = torch.randperm(8, device="cuda")  # int64
    rows = torch.empty(8, 64, dtype=torch.bfloat16, device="cuda")
    B = M.MOE_BF16
    q, s = torch.ones(8, 64, dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    y = torch.empty(8, 64, device="cuda")
    off = torch.tensor([0, 8], device="cuda")
    calls = [lambda i: M.moe_permute_rows(x, B, i, 4, 64, 2, 8, rows),
             lambda i: M.moe_permute_rows_backward(rows, B, i, 4, 64, 2, 8, x, B),
             lambda i: M.moe_combine_rows(rows, B, i, w, 4, 64, 2, 8, x, B),
             lambda i: M.moe_combine_rows_backward(x, B, rows, B, i, w, 4, 64, 2, 8, torch.empty_like(rows), None),
             lambda i: M.moe_matmul_i8(q, s, q, s, off if i.dtype == torch.int64 else off.int(), i, 8, 1, 8, 64, 8, 1,
                                       y, M.MOE_F32)]
    for call in calls:
        with pytest.raises(M.MoeError) as ei:
            call(inv)
        assert ei.value.status == M.MOE_ERR_INVALID_ARG and "int64" in ei.value.message
        call(inv.int())
