"""The routing's gradient (moe_route_backward) against its 64-bit definition; the
bounds count roundings (_block.py)."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

import _block
from _gpu import log

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
CODE = {F32: M.MOE_F32, BF16: M.MOE_BF16}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


def make(T, m, E, k, dtype, aux, seed=0):
    g = torch.Generator().manual_seed(seed + T + m + E)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(T=T, m=m, E=E, k=k, dtype=dtype)
    d["idx"] = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    d["w"], d["dw"] = torch.softmax(r(T, k), 1).cuda(), r(T, k).cuda()
    d["dl_add"] = 0.1 * r(T, E).cuda() if aux else None
    d["x"], d["dx_add"] = (r(T, m) + 0.2).to(dtype).cuda(), r(T, m).to(dtype).cuda()
    d["wr"] = (r(m, E) * m**-0.5).cuda()
    return d


class Guarded:
    def __init__(self, shape, dtype):
        n = 1
        for s in shape:
            n *= s
        self.buf = torch.full((n + 512,), 7.0, dtype=dtype, device="cuda")
        self.t = self.buf[256:256 + n].view(shape)
        self.t.fill_(NAN)

    def intact(self):
        assert bool((self.buf[:256] == 7).all()) and bool((self.buf[256 + self.t.numel():] == 7).all())


def call(d, dl, dx=None, dwr=None, db=None, ws=None, **other):
    v = {**d, **other}
    n = M.moe_route_backward_workspace_size(d["T"], d["m"], d["E"])
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
    M.moe_route_backward(v["dw"], v["idx"], v["w"], v["dl_add"], v["x"], CODE[d["dtype"]], v["wr"], v["dx_add"], d["T"],
                         d["m"], d["E"], d["k"], dl, dx, dwr, db, ws, n)


def outputs(d):
    T, m, E = d["T"], d["m"], d["E"]
    return [Guarded((T, E), F32), Guarded((T, m), d["dtype"]), Guarded((m, E), F32), Guarded((E,), F32)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,m,E,k,aux", [(1, 8, 1, 1, False), (1, 64, 8, 2, False), (3, 136, 2, 2, True), (65, 1000, 33, 4, True),
                                         (130, 264, 8, 2, False), (257, 4096, 16, 3, True), (64, 8200, 64, 8, False),
                                         (1111, 520, 5, 1, True), (5000, 128, 17, 2, False), (700, 2048, 64, 64, True), (8192, 64, 8, 2, False),
                                         (8193, 72, 4, 2, True), (20000, 136, 40, 3, False)])
def test_route_backward(T, m, E, k, aux, dtype):
    log(f"route gradient {dtype} T={T} m={m} E={E} k={k} aux={aux}")
    d = make(T, m, E, k, dtype, aux)
    outs = outputs(d)
    call(d, *(o.t for o in outs))
    torch.cuda.synchronize()
    want, bound = _block.route_backward(d["dw"], d["idx"], d["w"], d["dl_add"], d["x"], d["wr"], d["dx_add"], E, dtype)
    for name, o, w, b in zip(("d_logits", "dx", "dw_router", "db_router"), outs, want, bound):
        _block.check(o.t, w, b, name, log)
        o.intact()
    # parts: the same bits
    for keep in ((1,), (2,), (3,), ()):
        part = [torch.empty_like(o.t) if i in keep or i == 0 else None for i, o in enumerate(outs)]
        call(d, *part, **({} if 2 in keep else {"x": None}), **({} if 1 in keep else {"wr": None}))
        assert all(p is None or torch.equal(p, o.t) for p, o in zip(part, outs)), keep
    # dx over dx_add
    over = d["dx_add"].clone()
    call(d, torch.empty_like(outs[0].t), over, dx_add=over)
    assert torch.equal(over, outs[1].t)
    # without dx_add
    alone = torch.empty_like(outs[1].t)
    call(d, torch.empty_like(outs[0].t), alone, dx_add=None)
    want, bound = _block.route_backward(d["dw"], d["idx"], d["w"], d["dl_add"], d["x"], d["wr"], None, E, dtype)
    _block.check(alone, want[1], bound[1], "dx without dx_add", log)


def test_same_expert_twice_and_outside():
    """An expert named twice gets both parts; an index outside the experts reaches no logit."""
    d = make(50, 72, 6, 3, F32, False, seed=3)
    d["idx"][:20, 1] = d["idx"][:20, 0]
    d["idx"][30, 0], d["idx"][31, 2] = -1, 6
    d["idx"][32] = 1 << 30
    outs = outputs(d)
    call(d, *(o.t for o in outs))
    want, bound = _block.route_backward(d["dw"], d["idx"], d["w"], None, d["x"], d["wr"], d["dx_add"], 6, F32)
    for name, o, w, b in zip(("d_logits", "dx", "dw_router", "db_router"), outs, want, bound):
        _block.check(o.t, w, b, name, log)
    assert not bool(outs[0].t[32].any())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_non_finite_tokens_stay_alone(dtype):
    d = make(90, 136, 9, 2, dtype, True, seed=4)
    a, b = [o.t for o in outputs(d)], [o.t for o in outputs(d)]
    call(d, *a)
    d["dw"][7, 1] = NAN
    d["dx_add"][20, 3] = float("inf")
    call(d, *b)
    keep = [t for t in range(90) if t not in (7, 20)]
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1][keep], b[1][keep])
    assert not bool(torch.isfinite(b[1][7]).any()) and not bool(torch.isfinite(b[1][20, 3]))
    cols = [c for c in range(136) if c != 3]
    assert torch.equal(a[1][20][cols], b[1][20][cols])


def test_against_differences():
    """The gradient of sum(w * c) + sum(x * d) through logits, softmax over the choice, in 64 bits."""
    d = make(6, 16, 5, 3, F32, False, seed=5)
    x, wr, c, e = d["x"].double(), d["wr"].double(), d["dw"].double(), d["dx_add"].double()
    idx = d["idx"].long()
    loss = lambda x, wr, b: float((torch.softmax((x @ wr + b).gather(1, idx), 1) * c).sum() + (x * e).sum())  # noqa: E731
    d["w"] = torch.softmax((x @ wr).gather(1, idx), 1).float()
    outs = [o.t for o in outputs(d)]
    call(d, *outs)
    h, zero = 2.0**-13, torch.zeros(5, dtype=torch.float64, device="cuda")
    g = torch.Generator().manual_seed(6)
    for i, (base, grad) in enumerate([(x, outs[1]), (wr, outs[2]), (zero, outs[3])]):
        for at in torch.randperm(base.numel(), generator=g)[:10].tolist():
            v = [[x, wr, zero][j].clone() for j in range(3)]
            v[i].view(-1)[at] += h
            up = loss(*v)
            v[i].view(-1)[at] -= 2 * h
            want, got = (up - loss(*v)) / (2 * h), float(grad.reshape(-1)[at])
            # h^2 / 6 of a third derivative of order 20, 64-bit differences over h, fp32 gradients of order 1
            assert abs(got - want) <= 20 * h * h + 1e-11 / h + 1e-5 * (1 + abs(want)), (i, at, got, want)


def test_no_tokens():
    dwr, db = torch.full((64, 8), 3.0, device="cuda"), torch.full((8,), 3.0, device="cuda")
    M.moe_route_backward(None, None, None, None, None, M.MOE_BF16, None, None, 0, 64, 8, 2, None, None, dwr, db)
    assert not bool(dwr.any()) and not bool(db.any())


def test_graph_and_repeats():
    d = make(500, 1032, 33, 4, BF16, True, seed=7)
    a, b = [o.t for o in outputs(d)], [o.t for o in outputs(d)]
    n = M.moe_route_backward_workspace_size(500, 1032, 33)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    call(d, *a)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        call(d, *b, ws=ws)
    for _ in range(4):
        for t in b:
            t.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        d["dw"].mul_(0.75)
        call(d, *a)
        torch.cuda.synchronize()
