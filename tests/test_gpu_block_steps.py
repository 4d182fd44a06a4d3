"""A training step of a whole MoE block, operator by operator: what each left in memory against the
64-bit definition of what it found there, in bf16 and fp32.  The bounds count roundings (_block.py)."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

import _block
from _gpu import W_ABS, log
from test_gpu_add_norm import n64, reference
from test_gpu_block_chain import E, EPS, T, Block, k, m

pytestmark = pytest.mark.gpu

u = 2.0**-24
R = T * k


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_each_operator_of_a_step(dtype):
    b = Block(dtype, 3)
    b.step()
    torch.cuda.synchronize()
    i, w, o, U = b.inputs, b.leaves, b.o, _block.U[dtype]
    d = {n: t.double() for n, t in {**i, **w, **o}.items()}

    def check(name, want, bound):
        _block.check(o[name], want, bound, name, log)

    def rounded(want, bound):  # an output's bound: its rounding, of a value that is off by `bound` already
        return bound + U * (want.abs() + bound)

    # residual and norm
    s, _, rs, y, e_s, _, e_r, e_y = (None if v is None else torch.as_tensor(v).cuda() for v in reference(
        n64(i["x"]), n64(i["residual"]), n64(w["gamma"]), None, False, dtype))
    check("s", s, rounded(s, e_s))
    check("rstd", rs, e_r)
    check("y", y, rounded(y, e_y))
    # routing: a dot product of m terms and the bias; the experts of the largest logits; their softmax
    logits, size = d["y"] @ d["wr"] + d["br"], d["y"].abs() @ d["wr"].abs() + d["br"].abs()
    check("logits", logits, 2 * (m + 2) * u * size)
    idx = torch.topk(o["logits"], k, 1).indices
    assert torch.equal(o["idx"].long(), idx)
    gates = torch.softmax(d["logits"].gather(1, idx), 1)
    check("w", gates, torch.full_like(gates, W_ABS))
    # dispatch: assignment perm[r] is row r, its expert the one whose range holds r
    perm, flat = o["perm"].long(), idx.reshape(-1)
    assert torch.equal(perm.sort().values, torch.arange(R, device="cuda"))
    assert torch.equal(o["inv"].long()[perm], torch.arange(R, device="cuda"))
    assert torch.equal(flat[perm], torch.searchsorted(o["offsets"][1:].long(), torch.arange(R, device="cuda"), right=True))
    # experts
    where = (o["offsets"], o["perm"], k, R, dtype)
    want, bound = _block.forward(o["y"], w["wg"], w["wu"], w["wd"], *where)
    for name, v, e in zip(("rows", "gate", "up"), want, bound):
        check(name, v, e)
    # combine: a product and an addition for each of k rows
    rows = d["rows"][o["inv"].long().view(T, k)]
    terms = rows * d["w"][:, :, None]
    check("out", terms.sum(1), rounded(terms.sum(1), (k + 1) * u * terms.abs().sum(1)))
    # back: the rows' gradients and the gate weights'
    at = perm // k
    scaled = d["c"][at] * d["w"].view(-1)[perm][:, None]
    check("drows", scaled, rounded(scaled, u * scaled.abs()))
    terms = rows * d["c"][:, None]
    check("dw", terms.sum(2), (m + 1) * u * terms.abs().sum(2))
    want, bound = _block.backward(o["drows"], o["y"], w["wg"], w["wu"], w["wd"], o["gate"], o["up"], *where)
    for name, v, e in zip(("dxr", "dwg", "dwu", "dwd"), want, bound):
        check(name, v, e)
    terms = d["dxr"][o["inv"].long().view(T, k)]
    check("dxe", terms.sum(1), rounded(terms.sum(1), k * u * terms.abs().sum(1)))
    want, bound = _block.route_backward(o["dw"], o["idx"], o["w"], None, o["y"], w["wr"], o["dxe"], E, dtype)
    for name, v, e in zip(("dl", "dy", "dwr", "dbr"), want, bound):
        check(name, v, e)
    # residual norm's gradient: the bounds of test_gpu_add_norm.py
    r, v = d["rstd"][:, None], d["dy"] * d["gamma"]
    h = d["s"] * r
    a, aa = (v * h).mean(1, keepdim=True), (v * h).abs().mean(1, keepdim=True)
    part = r * (v - h * a)
    want = d["c"] + part
    e = r * (8 * u * (v.abs() + h.abs() * a.abs()) + (m + 6) * u * h.abs() * aa) + u * part.abs() + 2 * u * want.abs()
    check("dx", want, rounded(want, e))
    check("dgamma", (d["dy"] * h).sum(0), (T + 6) * u * (d["dy"] * h).abs().sum(0))
