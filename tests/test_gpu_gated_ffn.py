"""The gated feed-forward block on plain weights (moe_gated_ffn_forward, _backward)
against 64-bit definitions; the bounds count roundings (_block.py)."""
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


def inside(t):
    """t between NaNs: what is read beside it would show."""
    n = t.numel()
    buf = torch.full((n + 512,), NAN, dtype=t.dtype, device="cuda")
    buf[256:256 + n] = t.reshape(-1)
    return buf[256:256 + n].view(t.shape)


class Guarded:
    """An output between two guard zones that must stay as they were."""

    def __init__(self, shape, dtype, fill=7.0):
        n = 1
        for s in shape:
            n *= s
        self.buf = torch.full((n + 512,), 7.0, dtype=dtype, device="cuda")
        self.t = self.buf[256:256 + n].view(shape)
        self.t.fill_(fill)

    def intact(self):
        n = self.t.numel()
        assert bool((self.buf[:256] == 7).all()) and bool((self.buf[256 + n:] == 7).all())


def make(T, k, E, m, p, dtype, seed=0, only=None):
    """A block's tensors; k = 0: dense.  only: the experts that tokens choose from."""
    g = torch.Generator().manual_seed(seed + T * 7 + m * 3 + p)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = {"T": T, "k": max(1, k), "E": E, "m": m, "p": p, "rows": T * max(1, k), "dtype": dtype}
    d["x"] = inside((r(T, m) + 0.3).to(dtype).cuda())
    d["wg"], d["wu"] = (inside((r(E, m, p) * m**-0.5).to(dtype).cuda()) for _ in range(2))
    d["wd"] = inside((r(E, p, m) * p**-0.5).to(dtype).cuda())
    d["offsets"] = d["perm"] = None
    if k:
        pool = torch.tensor(list(range(E)) if only is None else only)
        idx = pool[torch.stack([torch.randperm(len(pool), generator=g)[:k] for _ in range(T)])] if T else torch.zeros(0, k)
        flat = idx.reshape(-1).long()
        d["perm"] = torch.sort(flat, stable=True).indices.to(torch.int32).cuda()
        c = torch.bincount(flat, minlength=E)
        d["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long), c.cumsum(0)]).to(torch.int32).cuda()
    R = d["rows"]
    d["gate"], d["up"] = (inside((r(R, p) * 1.5).to(dtype).cuda()) for _ in range(2))
    d["dy"] = inside(r(R, m).to(dtype).cuda())
    return d


def workspace(d, backward):
    n = M.moe_gated_ffn_workspace_size(CODE[d["dtype"]], d["rows"], d["m"], d["p"], d["E"], backward)
    return torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda"), n  # bytes 255: NaN in both types


def forward(d, y, gate=None, up=None, stream=None, ws=None):
    w, n = ws or workspace(d, 0)
    M.moe_gated_ffn_forward(d["x"], CODE[d["dtype"]], d["wg"], d["wu"], d["wd"], d["offsets"], d["perm"], d["T"], d["k"],
                            d["rows"], d["m"], d["p"], d["E"], y, gate, up, w, n, stream=stream)


def backward(d, dx, dwg, dwu, dwd, stream=None, ws=None):
    w, n = ws or workspace(d, 1)
    M.moe_gated_ffn_backward(d["dy"], d["x"], CODE[d["dtype"]], d["wg"], d["wu"], d["wd"], d["gate"], d["up"],
                             d["offsets"], d["perm"], d["T"], d["k"], d["rows"], d["m"], d["p"], d["E"], dx, dwg, dwu, dwd,
                             w, n, stream=stream)


def check_forward(d):
    y, gate, up = (Guarded((d["rows"], n), d["dtype"]) for n in (d["m"], d["p"], d["p"]))
    forward(d, y.t, gate.t, up.t)
    torch.cuda.synchronize()
    want, bound = _block.forward(d["x"], d["wg"], d["wu"], d["wd"], d["offsets"], d["perm"], d["k"], d["rows"], d["dtype"])
    for name, o, w, b in zip(("y", "gate", "up"), (y, gate, up), want, bound):
        _block.check(o.t, w, b, name, log)
        o.intact()
        if w.numel():
            assert bool((o.t[torch.isnan(w[:, 0])] == 7).all()), f"{name}: rows of no range"
    alone = Guarded((d["rows"], d["m"]), d["dtype"])
    forward(d, alone.t)
    assert torch.equal(alone.t, y.t)


def check_backward(d):
    R, E, m, p = d["rows"], d["E"], d["m"], d["p"]
    outs = [Guarded(s, d["dtype"]) for s in ((R, m), (E, m, p), (E, m, p), (E, p, m))]
    backward(d, *(o.t for o in outs))
    torch.cuda.synchronize()
    want, bound = _block.backward(d["dy"], d["x"], d["wg"], d["wu"], d["wd"], d["gate"], d["up"], d["offsets"], d["perm"],
                                  d["k"], R, d["dtype"])
    for name, o, w, b in zip(("dx", "dw_gate", "dw_up", "dw_down"), outs, want, bound):
        _block.check(o.t, w, b, name, log)
        o.intact()
    if R:
        assert bool((outs[0].t[torch.isnan(want[0][:, 0])] == 7).all()), "dx: rows of no range"


# T, k (0: dense), E, m, p, experts chosen from (None: all)
CASES = [(1, 0, 1, 8, 8, None), (1, 2, 8, 64, 128, None), (3, 2, 4, 72, 40, None), (5, 0, 1, 200, 136, None),
         (64, 2, 16, 264, 520, None), (130, 2, 3, 256, 512, None), (300, 2, 4, 320, 264, [0, 3]), (97, 3, 64, 136, 72, None),
         (333, 0, 1, 512, 1000, None), (40, 1, 5, 136, 1032, [2]), (700, 2, 3, 64, 24, None), (17, 0, 1, 1096, 64, None),
         (16, 0, 1, 512, 2048, None), (9, 2, 2, 2056, 128, None)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,m,p,only", CASES)
def test_forward(T, k, E, m, p, only, dtype):
    log(f"gated forward {dtype} T={T} k={k} E={E} m={m} p={p}")
    check_forward(make(T, k, E, m, p, dtype, only=only))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,m,p,only", CASES)
def test_backward(T, k, E, m, p, only, dtype):
    log(f"gated backward {dtype} T={T} k={k} E={E} m={m} p={p}")
    check_backward(make(T, k, E, m, p, dtype, seed=1, only=only))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("offsets", [[0, 10, 10, 60], [5, 20, 12, 90], [-4, 300, 7, 100], [0, 0, 0, 0], [200, 0, 50, 300]])
def test_any_offsets(offsets, dtype):
    """Gaps, empty experts, decreasing and wild offsets: read as clamped, other rows left alone."""
    log(f"gated offsets {offsets} {dtype}")
    d = make(50, 2, 3, 72, 136, dtype, seed=2)
    d["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    check_forward(d)
    check_backward(d)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_wild_permutation(dtype):
    """perm outside the tokens is clamped; the same token may fill many rows."""
    log(f"gated permutation {dtype}")
    d = make(30, 2, 2, 64, 72, dtype, seed=3)
    d["perm"][0], d["perm"][1], d["perm"][2:20] = -5, 1 << 30, 4
    check_forward(d)
    check_backward(d)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [20, 400])
def test_non_finite_rows_stay_alone(T, dtype):
    """A row with NaN or infinities changes its own results (and its expert's weight gradients) only."""
    log(f"gated non-finite rows {dtype} T={T}")
    d = make(T, 0, 1, 136, 72, dtype, seed=4)
    y = torch.empty(T, 136, dtype=dtype, device="cuda")
    forward(d, y)
    dx = torch.empty_like(y)
    backward(d, dx, None, None, None)
    bad = {3: NAN, T - 1: float("inf")}
    for r, v in bad.items():
        d["x"][r, 5] = v
        d["dy"][r, 7] = v
    y2, dx2 = torch.empty_like(y), torch.empty_like(y)
    forward(d, y2)
    backward(d, dx2, None, None, None)
    keep = [r for r in range(T) if r not in bad]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(dx[keep], dx2[keep])
    assert not bool(torch.isfinite(y2[list(bad)]).all(1).any()) and not bool(torch.isfinite(dx2[list(bad)]).all(1).any())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_rows_of_no_range_may_hold_anything(dtype):
    """Rows that no expert takes reach no weight gradient, NaN included."""
    d = make(60, 2, 3, 64, 136, dtype, seed=5)
    d["offsets"] = torch.tensor([0, 30, 70, 101], dtype=torch.int32, device="cuda")
    for n in ("dy", "gate", "up"):
        d[n][101:] = NAN
    check_backward(d)


@pytest.mark.parametrize("what", ["dx", "gate", "down"])
def test_parts_of_the_backward(what):
    """Each output without the others equals the full call's."""
    d = make(90, 2, 4, 136, 264, BF16, seed=6)
    full = [torch.zeros(s, dtype=BF16, device="cuda") for s in ((180, 136), (4, 136, 264), (4, 136, 264), (4, 264, 136))]
    backward(d, *full)
    keep = {"dx": (0,), "gate": (1, 2), "down": (3,)}[what]
    part = [torch.zeros_like(f) if i in keep else None for i, f in enumerate(full)]
    backward(d, *part)
    assert all(torch.equal(part[i], full[i]) for i in keep)


def test_dx_over_dy():
    d = make(100, 2, 4, 136, 264, BF16, seed=7)
    full = [torch.zeros(s, dtype=BF16, device="cuda") for s in ((200, 136), (4, 136, 264), (4, 136, 264), (4, 264, 136))]
    backward(d, *full)
    again = [d["dy"]] + [torch.zeros_like(f) for f in full[1:]]
    backward(d, *again)
    assert all(torch.equal(a, b) for a, b in zip(again, full))


def test_no_rows():
    """No tokens: the forward pass does nothing, the weight gradients are zeros."""
    d = make(4, 2, 3, 64, 72, F32, seed=8)
    w = [torch.full((3, 64, 72), 5.0, device="cuda"), torch.full((3, 64, 72), 5.0, device="cuda"),
         torch.full((3, 72, 64), 5.0, device="cuda")]
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    M.moe_gated_ffn_forward(None, M.MOE_F32, None, None, None, off, None, 0, 1, 0, 64, 72, 3, None)
    M.moe_gated_ffn_backward(None, None, M.MOE_F32, None, None, None, None, None, off, None, 0, 1, 0, 64, 72, 3, None, *w)
    assert all(not bool(t.any()) for t in w)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k", [(6, 2), (300, 2)])
def test_repeats_and_streams(T, k, dtype):
    """The same bits every time, on another stream, and from a replayed graph between eager calls."""
    d = make(T, k, 4, 136, 264, dtype, seed=9)
    R = d["rows"]
    shapes = ((R, 136), (R, 264), (R, 264)), ((R, 136), (4, 136, 264), (4, 136, 264), (4, 264, 136))
    first, other = ([[torch.zeros(s, dtype=dtype, device="cuda") for s in part] for part in shapes] for _ in range(2))
    ws = workspace(d, 0), workspace(d, 1)
    forward(d, *first[0], ws=ws[0])
    backward(d, *first[1], ws=ws[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        forward(d, *other[0], ws=ws[0])
        backward(d, *other[1], ws=ws[1])
    side.synchronize()
    assert all(torch.equal(a, b) for p, q in zip(first, other) for a, b in zip(p, q))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        forward(d, *other[0], ws=ws[0])
        backward(d, *other[1], ws=ws[1])
    for i in range(4):
        for p in other:
            for t in p:
                t.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for p, q in zip(first, other) for a, b in zip(p, q)), i
        d["x"].mul_(1.25)  # new inputs in place
        forward(d, *first[0])
        backward(d, *first[1])


def test_gradient_against_differences():
    """fp32: the gradients of sum(y * c) against central differences of the forward pass in 64 bits."""
    d = make(5, 2, 3, 16, 24, F32, seed=10)
    R = d["rows"]
    y, gate, up = torch.empty(R, 16, device="cuda"), torch.empty(R, 24, device="cuda"), torch.empty(R, 24, device="cuda")
    forward(d, y, gate, up)
    d["gate"], d["up"] = gate, up
    outs = [torch.zeros(s, device="cuda") for s in ((R, 16), (3, 16, 24), (3, 16, 24), (3, 24, 16))]
    backward(d, *outs)
    c = d["dy"].double()
    dx = torch.zeros(5, 16, dtype=torch.float64, device="cuda").index_add_(0, d["perm"].long() // 2, outs[0].double())
    grads = dict(x=dx, wg=outs[1], wu=outs[2], wd=outs[3])
    h = 2.0**-12
    g = torch.Generator().manual_seed(11)
    for name, grad in grads.items():
        base = {n: d[n].double() for n in grads}
        for at in torch.randperm(base[name].numel(), generator=g)[:12].tolist():
            ends = []
            for sign in (1, -1):
                v = {n: t.clone() for n, t in base.items()}
                v[name].view(-1)[at] += sign * h
                (out, _, _), _ = _block.forward(v["x"], v["wg"], v["wu"], v["wd"], d["offsets"], d["perm"], 2, R, F32)
                ends.append(float((out * c).sum()))
            want, got = (ends[0] - ends[1]) / (2 * h), float(grad.reshape(-1)[at])
            # h^2 / 6 of a third derivative of order 10, 64-bit differences over h, fp32 gradients of order 1
            assert abs(got - want) <= h * h * 10 + 1e-10 / h + 1e-5 * (1 + abs(want)), (name, at, got, want)


@pytest.mark.parametrize("op", ["forward", "backward"])
@pytest.mark.parametrize("T,m,p,split", [(2523, 8192, 64, None), (2400, 64, 8192, None), (2500, 8192, 64, 1000), (2300, 64, 8192, 530)])
def test_rounds_of_large_tiles(T, m, p, split, op):
    """Ten row blocks by 32 (or 64) column blocks of 256 x 256 tiles, 1.25 (2.5) rounds of 256: the last round's
    are cut in two, the halves of a short row block among them."""
    log(f"gated {op} T={T} m={m} p={p}")
    d = make(T, 0, 1, m, p, BF16, seed=12) if split is None else make(T, 1, 2, m, p, BF16, seed=12)
    if split:
        d["offsets"] = torch.tensor([0, split, T], dtype=torch.int32, device="cuda")
    check_forward(d) if op == "forward" else check_backward(d)


def test_weight_gradients_split_over_their_rows():
    """Few tiles and many rows: the rows are shared and the parts joined, each expert's by its own count."""
    for dtype in (BF16, F32):
        d = make(3000, 1, 3, 136, 72, dtype, seed=13)
        d["offsets"] = torch.tensor([0, 2500, 2500, 2990], dtype=torch.int32, device="cuda")
        check_backward(d)
