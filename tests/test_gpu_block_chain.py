"""A whole MoE block of a training step through the operators, forwards and back,
against torch's automatic differentiation in 64 bits; captured and replayed."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

from _gpu import F32_REL, log

pytestmark = pytest.mark.gpu

T, E, k, m, p, EPS = 70, 5, 2, 192, 264, 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


class Block:
    """One block's tensors and its step: loss = sum(out * c) with out = s + MoE(norm(s)), s = x + residual."""

    def __init__(self, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
        self.code, self.dtype = (M.MOE_F32 if dtype == torch.float32 else M.MOE_BF16), dtype
        self.inputs = dict(x=r(T, m).to(dtype), residual=r(T, m).to(dtype), c=r(T, m).to(dtype))
        self.leaves = dict(gamma=1 + 0.2 * r(m), wr=r(m, E) * m**-0.5, br=0.1 * r(E), wg=(r(E, m, p) * m**-0.5).to(dtype),
                           wu=(r(E, m, p) * m**-0.5).to(dtype), wd=(r(E, p, m) * p**-0.5).to(dtype))
        n = lambda *s, t=dtype: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        f, i = torch.float32, torch.int32
        self.o = dict(s=n(T, m), y=n(T, m), rstd=n(T, t=f), logits=n(T, E, t=f), idx=n(T, k, t=i), w=n(T, k, t=f), counts=n(E, t=i),
                      offsets=n(E + 1, t=i), perm=n(T * k, t=i), inv=n(T * k, t=i), rows=n(T * k, m), gate=n(T * k, p),
                      up=n(T * k, p), out=n(T, m), drows=n(T * k, m), dw=n(T, k, t=f), dxr=n(T * k, m), dwg=n(E, m, p),
                      dwu=n(E, m, p), dwd=n(E, p, m), dxe=n(T, m), dl=n(T, E, t=f), dy=n(T, m), dwr=n(m, E, t=f), dbr=n(E, t=f),
                      dx=n(T, m), dgamma=n(m, t=f))
        sizes = [M.moe_gated_ffn_workspace_size(self.code, T * k, m, p, E, b) for b in (0, 1)]
        sizes += [M.moe_route_backward_workspace_size(T, m, E), M.moe_norm_backward_workspace_size(T, m)]
        self.ws_bytes = max(sizes)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device="cuda")

    def step(self):
        i, w, o, c = self.inputs, self.leaves, self.o, self.code
        R, ws, n = T * k, self.ws, self.ws_bytes
        M.moe_add_norm_forward(i["x"], i["residual"], c, M.MOE_NORM_RMS, w["gamma"], None, EPS, T, m, o["s"], o["y"], rstd=o["rstd"])
        M.moe_route_topk(o["y"], c, w["wr"], w["br"], T, m, E, k, 0, o["logits"], o["idx"], o["w"])
        M.moe_dispatch(o["idx"], T, E, k, o["counts"], o["offsets"], o["perm"], o["inv"])
        where = (o["offsets"], o["perm"], T, k, R, m, p, E)
        M.moe_gated_ffn_forward(o["y"], c, w["wg"], w["wu"], w["wd"], *where, o["rows"], o["gate"], o["up"], ws, n)
        M.moe_combine_rows(o["rows"], c, o["inv"], o["w"], T, m, k, R, o["out"], c)
        # back, from d out = c (the residual stream adds c to d s as well)
        M.moe_combine_rows_backward(i["c"], c, o["rows"], c, o["inv"], o["w"], T, m, k, R, o["drows"], o["dw"])
        M.moe_gated_ffn_backward(o["drows"], o["y"], c, w["wg"], w["wu"], w["wd"], o["gate"], o["up"], *where, o["dxr"], o["dwg"],
                                 o["dwu"], o["dwd"], ws, n)
        M.moe_permute_rows_backward(o["dxr"], c, o["inv"], T, m, k, R, o["dxe"], c)
        M.moe_route_backward(o["dw"], o["idx"], o["w"], None, o["y"], c, w["wr"], o["dxe"], T, m, E, k, o["dl"], o["dy"], o["dwr"],
                             o["dbr"], ws, n)
        M.moe_add_norm_backward(o["dy"], i["c"], o["s"], c, M.MOE_NORM_RMS, w["gamma"], None, o["rstd"], T, m, o["dx"], o["dgamma"],
                                None, ws, n)


def reference(b):
    """Loss gradients of the same block in 64 bits, with the step's own choice of experts."""
    v = {n: t.double().requires_grad_() for n, t in {**b.inputs, **b.leaves}.items()}
    s = v["x"] + v["residual"]
    y = s * (s.square().mean(1, keepdim=True) + EPS).rsqrt() * v["gamma"]
    idx = b.o["idx"].long()
    w = torch.softmax((y @ v["wr"] + v["br"]).gather(1, idx), 1)
    h = torch.nn.functional.silu(torch.einsum("tm,emp->tep", y, v["wg"])) * torch.einsum("tm,emp->tep", y, v["wu"])
    rows = torch.einsum("tep,epm->tem", h, v["wd"]).gather(1, idx[:, :, None].expand(-1, -1, m))
    moe = (rows * w[:, :, None]).sum(1)
    ((s + moe) * v["c"].detach()).sum().backward()
    return moe.detach(), {n: v[n].grad for n in ("x", "residual", *b.leaves)}


def test_training_step():
    b = Block(torch.float32)
    b.step()
    torch.cuda.synchronize()
    moe, grads = reference(b)
    got = dict(moe=b.o["out"], x=b.o["dx"], residual=b.o["dx"], gamma=b.o["dgamma"], wr=b.o["dwr"], br=b.o["dbr"], wg=b.o["dwg"],
               wu=b.o["dwu"], wd=b.o["dwd"])
    for name, want in {"moe": moe, **grads}.items():
        err, scale = float((got[name].double() - want).abs().max()), float(want.abs().max())
        log(f"  {name}: max|err| {err:.3e} of {scale:.3e}")
        assert err <= F32_REL * scale, name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_captured_step(dtype):
    """The step's bits from a graph that is replayed between eager steps on new inputs."""
    a, b = Block(dtype, 1), Block(dtype, 1)
    a.step()
    b.step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        b.step()
    for turn in range(4):
        for t in b.o.values():
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for n in a.o:
            assert torch.equal(a.o[n], b.o[n]), (turn, n)
        for blk in (a, b):
            blk.inputs["x"].mul_(-0.75)
            blk.leaves["wg"].mul_(1.25)
        a.step()
        torch.cuda.synchronize()
