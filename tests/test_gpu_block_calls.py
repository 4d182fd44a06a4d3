"""Calls of the trainable block that its documentation allows beside the usual ones: a permutation
without offsets, outputs alone where rows come in two parts or reductions are split, outputs over
inputs there, two calls at once, and graphs that share a workspace."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

import _block
from _gpu import log
from test_gpu_add_norm import EPS, rnd
from test_gpu_gated_ffn import BF16, CODE, F32, Guarded, backward, check_backward, check_forward, forward, make, workspace

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


@BOTH
@pytest.mark.parametrize("T,k", [(7, 2), (110, 3), (1, 5)])
def test_permutation_without_offsets(T, k, dtype):
    """One expert takes all rows, in the permutation's order."""
    log(f"gated, perm without offsets, {dtype} T={T} k={k}")
    d = make(T, 0, 1, 136, 264, dtype, seed=20)
    g = torch.Generator().manual_seed(21)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    R = T * k
    d.update(k=k, rows=R, perm=torch.randperm(R, generator=g).to(torch.int32).cuda(), gate=r(R, 264), up=r(R, 264), dy=r(R, 136))
    check_forward(d)
    check_backward(d)


# few rows: two bf16 parts, split reductions; 90 rows an expert: one part; 1000: split weight gradients
SIZES = [(9, 2, 2, 1032, 520), (90, 2, 2, 264, 520), (1000, 1, 1, 136, 72)]


@BOTH
@pytest.mark.parametrize("T,k,E,m,p", SIZES)
def test_outputs_alone_and_over_inputs(T, k, E, m, p, dtype):
    d = make(T, k, E, m, p, dtype, seed=22)
    R = d["rows"]
    shapes = ((R, m), (E, m, p), (E, m, p), (E, p, m))
    full = [torch.zeros(s, dtype=dtype, device="cuda") for s in shapes]
    backward(d, *full)
    for keep in ((0,), (1, 2), (3,), (0, 3), (1, 2, 3)):
        part = [Guarded(s, dtype) if i in keep else None for i, s in enumerate(shapes)]
        backward(d, *(o.t if o else None for o in part))
        torch.cuda.synchronize()
        for o, f in zip(part, full):
            if o:
                assert torch.equal(o.t, f), keep
                o.intact()
    again = [d["dy"].clone()] + [torch.zeros_like(f) for f in full[1:]]
    backward({**d, "dy": again[0]}, *again)  # dx over dy
    assert all(torch.equal(a, b) for a, b in zip(again, full))


@BOTH
@pytest.mark.parametrize("T,k,E,m,p", SIZES)
def test_two_calls_at_once(T, k, E, m, p, dtype):
    """Two blocks on two streams with a workspace each: each has its own results."""
    blocks = [make(T, k, E, m, p, dtype, seed=s) for s in (23, 24)]

    def outputs(d):
        R = d["rows"]
        return ([torch.zeros(s, dtype=dtype, device="cuda") for s in ((R, m), (R, p), (R, p))],
                [torch.zeros(s, dtype=dtype, device="cuda") for s in ((R, m), (E, m, p), (E, m, p), (E, p, m))])

    want, got = [outputs(d) for d in blocks], [outputs(d) for d in blocks]
    for d, (f, b) in zip(blocks, want):
        forward(d, *f)
        backward(d, *b)
    spaces = [(workspace(d, 0), workspace(d, 1)) for d in blocks]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(3):
        for d, (f, b), (wf, wb), s in zip(blocks, got, spaces, streams):
            forward(d, *f, stream=s, ws=wf)
            backward(d, *b, stream=s, ws=wb)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for p_, q in zip(w, g) for a, b in zip(p_, q))


@BOTH
def test_graphs_that_share_a_workspace(dtype):
    """Replayed in turn, with eager calls in the same workspace between them."""
    blocks = [make(40, 2, 3, 520, 264, dtype, seed=25), make(9, 2, 3, 1032, 136, dtype, seed=26)]
    n = max(M.moe_gated_ffn_workspace_size(CODE[dtype], d["rows"], d["m"], d["p"], d["E"], b) for d in blocks for b in (0, 1))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda"), n
    new = lambda d: [torch.zeros(s, dtype=dtype, device="cuda") for s in (  # noqa: E731
        (d["rows"], d["m"]), (d["rows"], d["m"]), (3, d["m"], d["p"]), (3, d["m"], d["p"]), (3, d["p"], d["m"]))]

    def step(d, o):
        forward(d, o[0], ws=ws)
        backward(d, *o[1:], ws=ws)

    want, got = [new(d) for d in blocks], [new(d) for d in blocks]
    for d, o in zip(blocks, got):  # loads the kernels before the capture
        step(d, o)
    torch.cuda.synchronize()
    graphs, side = [], torch.cuda.Stream()
    for d, o in zip(blocks, got):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(d, o)
        graphs.append(graph)
    for turn in range(4):
        for o in got:
            for t in o:
                t.fill_(float("nan"))
        for g in graphs[::1 if turn % 2 else -1]:
            g.replay()
        for d, o in zip(blocks, want):
            step(d, o)
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, g)), turn
        for d in blocks:
            d["x"].mul_(-1.25)
            d["dy"].mul_(0.75)


@BOTH
@pytest.mark.parametrize("T,m", [(1, 8), (5, 264), (777, 2048), (50, 9000)])
def test_residual_norm_in_place_with_codes(T, m, dtype):
    """sum and y over the inputs, with codes; and a residual that is x itself."""
    x, r, gamma, beta = rnd((T, m), dtype, 1), rnd((T, m), dtype, 2, 3.0), rnd((m,), F32, 3, 0.2, 1.0), rnd((m,), F32, 4, 0.3)

    def call(x, r, s, y):
        o = dict(codes=torch.empty(T, m, dtype=torch.int8, device="cuda"), scale=torch.empty(T, device="cuda"),
                 mean=torch.empty(T, device="cuda"), rstd=torch.empty(T, device="cuda"))
        M.moe_add_norm_forward(x, r, CODE[dtype], M.MOE_NORM_LAYER, gamma, beta, EPS, T, m, s, y, **o)
        return s, y, *o.values()

    want = call(x, r, torch.empty_like(x), torch.empty_like(x))
    a, b = x.clone(), r.clone()
    assert all(torch.equal(p, q) for p, q in zip(call(a, b, b, a), want))
    a, b = x.clone(), r.clone()
    assert all(torch.equal(p, q) for p, q in zip(call(a, b, a, b), want))
    twice = call(x, x, torch.empty_like(x), torch.empty_like(x))
    a = x.clone()
    assert all(torch.equal(p, q) for p, q in zip(call(a, a, a, torch.empty_like(a)), twice))
    assert torch.equal(twice[0], (2 * x.float()).to(dtype))


@BOTH
def test_routing_gradient_over_its_inputs(dtype):
    """dx over x without the weight gradient, d_router over w_router, d_logits from the loss alone."""
    T, m, E, k = 333, 264, 12, 3
    g = torch.Generator().manual_seed(27)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    w, dw, aux = torch.softmax(r(T, k), 1), r(T, k), 0.1 * r(T, E)
    x, add, wr = r(T, m).to(dtype), r(T, m).to(dtype), r(m, E) * m**-0.5
    n = M.moe_route_backward_workspace_size(T, m, E)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def call(dw, x, wr, add, dx, dwr, db):
        dl = torch.empty(T, E, device="cuda")
        M.moe_route_backward(dw, idx, w, aux, x, CODE[dtype], wr, add, T, m, E, k, dl, dx, dwr, db, ws, n)
        return dl

    dx, dwr, db = torch.empty_like(x), torch.empty_like(wr), torch.empty(E, device="cuda")
    dl = call(dw, x, wr, add, dx, dwr, db)
    a, b = x.clone(), torch.empty_like(db)
    assert torch.equal(call(dw, a, wr, add, a, None, b), dl) and torch.equal(a, dx) and torch.equal(b, db)
    v = wr.clone()
    a = torch.empty_like(dx)
    assert torch.equal(call(dw, x, v, add, a, v, None), dl) and torch.equal(v, dwr) and torch.equal(a, dx)
    none = call(torch.zeros_like(dw), None, None, None, None, None, b)
    assert torch.equal(none, aux)
    _block.check(b, aux.double().sum(0), 2 * (T + 1) * _block.u * aux.double().abs().sum(0), "db_router of the loss alone", log)
