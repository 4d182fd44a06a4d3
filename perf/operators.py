"""The row operators around an MoE layer's experts, as cases to be timed and compared.

Four kinds of call: the layer's input norm (forward, and backward with the weight
gradients), rows sorted by expert and their gradient, expert rows combined back to their
tokens with the gate weights and that step's gradient, and the int8 product with a scale
per token and per output channel, dense or over the experts' row ranges.

``run`` computes each in elementary torch operations in 32 bits; with ``own`` set it makes
the calls of mixture_experts_layer_gemv_amd.  ``exact`` computes the same from the
definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---- cases ------------------------------------------------------------------------


def _norm(name, op, norm, dtype, T, m):
    return {"name": name, "op": op, "norm": norm, "dtype": dtype, "T": T, "m": m}


def _rows(name, op, T, k, E, m, dtype, rows, drop=0.0):
    return {"name": name, "op": op, "T": T, "k": k, "E": E, "m": m, "dtype": dtype, "rows": rows, "drop": drop}


def _product(name, T, k, E, K, N, out):
    return {"name": name, "op": "product", "T": T, "k": k, "E": E, "K": K, "N": N, "out": out}


def listed():
    return [
        # one decode step of the Mixtral-shaped layer: a launch's latency is what counts
        _norm("norm_rms_decode", "norm", "rms", "bf16", 16, 4096),
        # its prefill batch: the row streams in and out once
        _norm("norm_layer_prefill", "norm", "layer", "bf16", 8192, 4096),
        # the same batch in training: gradients of the rows, gamma and beta
        _norm("norm_layer_grad_prefill", "norm_grad", "layer", "bf16", 8192, 4096),
        # a ragged fp32 batch whose row is no power of two
        _norm("norm_rms_grad_ragged", "norm_grad", "rms", "f32", 777, 5000),
        # a prefill batch copied into expert order
        _rows("sort_prefill", "sort", 8192, 2, 8, 4096, "bf16", "bf16"),
        # the gradient of that step with assignments dropped for capacity, four experts a token
        _rows("sort_grad_ragged", "sort_grad", 1237, 4, 16, 1000, "f32", "f32", 0.1),
        # decode: the experts' fp32 rows back to their tokens
        _rows("combine_decode", "combine", 64, 2, 8, 4096, "bf16", "f32"),
        # its gradient over a training batch: expert rows' and gate weights'
        _rows("combine_grad_prefill", "combine_grad", 8192, 2, 16, 4096, "bf16", "bf16"),
        # a dense int8 projection for sixteen tokens: the weights stream once
        _product("product_decode", 16, 0, 1, 4096, 14336, "bf16"),
        # the experts' up projection at decode, rows gathered through the permutation
        _product("product_experts_decode", 64, 2, 8, 4096, 14336, "bf16"),
        # a ragged dense batch, fp32 out
        _product("product_ragged", 1003, 0, 1, 6400, 4096, "f32"),
        # the experts' up projection at prefill
        _product("product_experts_prefill", 8192, 2, 8, 4096, 14336, "bf16"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "sort", "sort_grad", "combine", "combine_grad", "product", "product"])
    if op in ("norm", "norm_grad"):
        m = _log(rng, 64, 16384, 8)
        return {"op": op, "norm": rng.choice(["layer", "rms"]), "dtype": rng.choice(["bf16", "f32"]),
                "T": _log(rng, 1, min(16384, (1 << 25) // (2 * m))), "m": m}
    E = rng.choice([1, 2, 8, 12, 16, 33, 64])
    k = min(E, rng.choice([1, 2, 2, 3, 4, 6, 8]))
    if op == "product":
        k = rng.choice([0, k]) if E == 1 else k
        K, N = _log(rng, 128, 14336, 16), _log(rng, 128, 14336, 16)
        most = min(8192 * 2, (1 << 39) // (K * N))
        while E * K * N > 1 << 29:
            E = (E + 1) // 2
        k = min(E, k)
        return {"op": op, "T": max(1, _log(rng, 1, most) // max(1, k)), "k": k, "E": E, "K": K, "N": N,
                "out": rng.choice(["bf16", "f32"])}
    m = _log(rng, 64, 8192, 8)
    return {"op": op, "T": _log(rng, 1, min(8192, (1 << 25) // (k * m))), "k": k, "E": E, "m": m,
            "dtype": rng.choice(["bf16", "f32"]), "rows": rng.choice(["bf16", "f32"]) if op.startswith("combine") else "",
            "drop": rng.choice([0.0, 0.0, 0.1, 0.7])}


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        T, m, s = case["T"], case["m"], SIZE[case["dtype"]]
        wide = 1 if case["norm"] == "rms" else 2  # gamma (and beta); rstd (and mean)
        if op == "norm":
            return {"bytes": 2 * T * m * s + 4 * wide * (m + T), "flops": 8 * T * m}
        return {"bytes": 3 * T * m * s + 4 * m + 4 * wide * (m + T), "flops": 16 * T * m}
    T, k = case["T"], case["k"]
    if op == "product":
        R, E, K, N = T * max(1, k), case["E"], case["K"], case["N"]
        used = min(E, R)
        index = 4 * (E + 1) + 4 * R if k else 0
        return {"bytes": T * K + 4 * T + used * N * (K + 4) + R * N * SIZE[case["out"]] + index, "flops": 2 * R * K * N}
    m, s = case["m"], SIZE[case["dtype"]]
    kept = T * k - int(case["drop"] * T * k)
    r = SIZE[case["rows"] or case["dtype"]]
    if op in ("sort", "sort_grad"):
        return {"bytes": T * m * s + kept * m * r + 4 * T * k, "flops": kept * m}
    if op == "combine":
        return {"bytes": T * m * s + kept * m * r + 8 * T * k, "flops": 2 * kept * m}
    return {"bytes": T * m * s + 2 * kept * m * r + 12 * T * k, "flops": 4 * kept * m}


# ---- inputs -----------------------------------------------------------------------


def _activations(g, T, m, dtype):
    """Rows as a residual stream has them: unit scale, an offset per channel, a few loud channels."""
    x = torch.randn(T, m, generator=g, device="cuda")
    loud = torch.where(torch.rand(m, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    x.mul_(loud).add_(0.3 * torch.randn(m, generator=g, device="cuda"))
    return x.to(DTYPES[dtype])


def _choices(g, T, k, E):
    """k different experts for each token, some experts more popular than others."""
    score = torch.rand(T, E, generator=g, device="cuda").clamp_min(1e-9).log().neg().log().neg()
    return torch.topk(score - 0.5 * torch.arange(1, E + 1, device="cuda").log(), k, dim=1).indices


def _plan(idx, keep):
    """The dispatch of top-k choices: rows in expert order, in order of assignment within an expert; an assignment that is not kept
    has no row (its place is -1).  Returns each assignment's row, each row's assignment and the experts' row ranges."""
    a = idx.reshape(-1)
    order = torch.sort(torch.where(keep, a, a.max() + 1), stable=True).indices
    rows = int(keep.sum())
    perm = order[:rows]
    inv = torch.full_like(a, -1)
    inv[perm] = torch.arange(rows, device=a.device)
    return inv.to(torch.int32), perm.to(torch.int32), rows


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op in ("norm", "norm_grad"):
        T, m, dt = case["T"], case["m"], DTYPES[case["dtype"]]
        s["x"] = _activations(g, T, m, case["dtype"])
        s["gamma"] = 1 + 0.2 * torch.randn(m, generator=g, device="cuda")
        s["beta"] = 0.1 * torch.randn(m, generator=g, device="cuda") if case["norm"] == "layer" else None
        if op == "norm":
            s["y"] = torch.empty_like(s["x"])
            s["mean"] = torch.empty(T, device="cuda") if case["norm"] == "layer" else None
            s["rstd"] = torch.empty(T, device="cuda")
            return s
        # what the forward pass saved
        x = s["x"].double()
        mean = x.mean(1) if case["norm"] == "layer" else torch.zeros(T, dtype=torch.float64, device="cuda")
        s["rstd"] = ((x - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        s["mean"] = mean.float() if case["norm"] == "layer" else None
        s["dy"] = torch.randn(T, m, generator=g, device="cuda").to(dt)
        s["dx"] = torch.empty_like(s["x"])
        s["dgamma"] = torch.empty(m, device="cuda")
        s["dbeta"] = torch.empty(m, device="cuda") if case["norm"] == "layer" else None
        if own:
            import mixture_experts_layer_gemv_amd as M

            s["bytes"] = M.moe_norm_backward_workspace_size(T, m)
            s["workspace"] = torch.empty(max(256, s["bytes"]), dtype=torch.uint8, device="cuda")
        return s
    T, k, E = case["T"], case["k"], case["E"]
    if op == "product":
        K, N = case["K"], case["N"]
        x = _activations(g, T, K, "f32")
        s["x_scale"] = x.abs().amax(1).clamp_min(1e-20) / 127
        s["x"] = torch.round(x / s["x_scale"][:, None]).to(torch.int8)
        w = torch.randn(E, N, K, generator=g, device="cuda")
        s["w_scale"] = w.abs().amax(2) * (0.02 / 127)
        s["w"] = w.mul_((0.02 / s["w_scale"])[:, :, None]).round_().to(torch.int8)
        del w
        s["rows"] = T * max(1, k)
        s["offsets"] = s["perm"] = None
        if k:
            idx = _choices(g, T, k, E)
            _, s["perm"], _ = _plan(idx, torch.ones(T * k, dtype=torch.bool, device="cuda"))
            counts = torch.bincount(idx.reshape(-1), minlength=E)
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
            s["most"] = int(counts.max())  # rows that the fullest expert takes
        s["y"] = torch.empty(s["rows"], N, dtype=DTYPES[case["out"]], device="cuda")
        return s
    m = case["m"]
    idx = _choices(g, T, k, E)
    score = torch.rand(T * k, generator=g, device="cuda")
    keep = torch.ones(T * k, dtype=torch.bool, device="cuda")
    keep[torch.sort(score).indices[: int(case["drop"] * T * k)]] = False
    s["inv"], s["perm"], s["rows"] = _plan(idx, keep)
    dt, rt = DTYPES[case["dtype"]], DTYPES[case["rows"] or case["dtype"]]
    s["w"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
    if op in ("sort", "combine_grad"):
        s["x"] = _activations(g, T, m, case["dtype"])
    if op != "sort":
        s["r"] = torch.randn(s["rows"], m, generator=g, device="cuda").to(rt)
    if op in ("sort", "combine_grad"):
        s["out"] = torch.empty(s["rows"], m, dtype=rt, device="cuda")
        s["dw"] = torch.empty(T, k, device="cuda")
    else:
        s["out"] = torch.empty(T, m, dtype=dt, device="cuda")
    return s


# ---- one pass ---------------------------------------------------------------------


def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "sort": _plain_sort, "sort_grad": _plain_sort_grad,
            "combine": _plain_combine, "combine_grad": _plain_combine_grad, "product": _plain_product}[s["op"]](s)


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1) if s["case"]["norm"] == "layer" else None
    d = x - mean[:, None] if mean is not None else x
    rstd = (d.square().mean(1) + EPS).rsqrt()
    y = d * rstd[:, None] * s["gamma"]
    if s["beta"] is not None:
        y = y + s["beta"]
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_grad(s):
    x, dy = s["x"].float(), s["dy"].float()
    hat = (x - s["mean"][:, None] if s["mean"] is not None else x) * s["rstd"][:, None]
    g = dy * s["gamma"]
    dx = g - hat * (g * hat).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * s["rstd"][:, None]
    return dx.to(s["x"].dtype), (dy * hat).sum(0), dy.sum(0) if s["mean"] is not None else None


def _plain_sort(s):
    return s["x"][(s["perm"] // s["case"]["k"]).long()]


def _gather(rows, inv):
    """Each assignment's row in 32 bits; zeros where it has none."""
    r = rows.float()
    there = inv >= 0
    if not len(r):
        return r.new_zeros(len(inv), r.shape[1])
    return torch.where(there[:, None], r[inv.clamp_min(0).long()], 0.0)


def _plain_sort_grad(s):
    c = s["case"]
    return _gather(s["r"], s["inv"]).view(c["T"], c["k"], c["m"]).sum(1).to(s["out"].dtype)


def _plain_combine(s):
    c = s["case"]
    return (_gather(s["r"], s["inv"]).view(c["T"], c["k"], c["m"]) * s["w"][:, :, None]).sum(1).to(s["out"].dtype)


def _plain_combine_grad(s):
    c = s["case"]
    dy = s["x"].float()
    dw = (_gather(s["r"], s["inv"]).view(c["T"], c["k"], c["m"]) * dy[:, None, :]).sum(2)
    a = s["perm"].long()
    return (dy[a // c["k"]] * s["w"].view(-1)[a][:, None]).to(s["r"].dtype), dw


def _plain_product(s):
    c = s["case"]
    x = s["x"].float()
    if s["perm"] is None:
        y = (x @ s["w"][0].float().t()) * s["x_scale"][:, None] * s["w_scale"][0]
        return y.to(s["y"].dtype)
    token = (s["perm"] // c["k"]).long()
    at = torch.arange(s["rows"], device=x.device)
    expert = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    place = at - s["offsets"].long()[expert]
    padded = x.new_zeros(c["E"], s["most"], c["K"])
    padded[expert, place] = x[token]
    y = torch.bmm(padded, s["w"].float().transpose(1, 2).contiguous())[expert, place]
    return (y * s["x_scale"][token][:, None] * s["w_scale"][expert]).to(s["y"].dtype)


def _own(s):
    import mixture_experts_layer_gemv_amd as M

    c, op = s["case"], s["op"]
    code = {torch.float32: M.MOE_F32, torch.bfloat16: M.MOE_BF16}
    if op in ("norm", "norm_grad"):
        T, m, dt, kind = c["T"], c["m"], code[s["x"].dtype], M.MOE_NORM_LAYER if c["norm"] == "layer" else M.MOE_NORM_RMS
        if op == "norm":
            M.moe_norm_forward(s["x"], dt, kind, s["gamma"], s["beta"], EPS, T, m, s["y"], s["mean"], s["rstd"])
            return s["y"], s["mean"], s["rstd"]
        M.moe_norm_backward(s["dy"], s["x"], dt, kind, s["gamma"], s["mean"], s["rstd"], T, m, s["dx"], s["dgamma"],
                            s["dbeta"], s["workspace"], s["bytes"])
        return s["dx"], s["dgamma"], s["dbeta"]
    T, k = c["T"], c["k"]
    if op == "product":
        M.moe_matmul_i8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["offsets"], s["perm"], T, max(1, k), s["rows"],
                        c["K"], c["N"], c["E"], s["y"], code[s["y"].dtype])
        return s["y"]
    m, rows, out = c["m"], s["rows"], s["out"]
    if op == "sort":
        M.moe_permute_rows(s["x"], code[s["x"].dtype], s["inv"], T, m, k, rows, out)
    elif op == "sort_grad":
        M.moe_permute_rows_backward(s["r"], code[s["r"].dtype], s["inv"], T, m, k, rows, out, code[out.dtype])
    elif op == "combine":
        M.moe_combine_rows(s["r"], code[s["r"].dtype], s["inv"], s["w"], T, m, k, rows, out, code[out.dtype])
    else:
        M.moe_combine_rows_backward(s["x"], code[s["x"].dtype], s["r"], code[s["r"].dtype], s["inv"], s["w"], T, m, k,
                                    rows, out, s["dw"])
        return out, s["dw"]
    return out


# ---- the definitions in 64 bits -----------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        n = x.shape[1]
        mean = x.sum(1) / n if case["norm"] == "layer" else x.new_zeros(len(x))
        var = torch.einsum("tm,tm->t", x - mean[:, None], x - mean[:, None]) / n
        rstd = 1 / torch.sqrt(var + EPS)
        y = torch.addcmul(s["beta"].double() if s["beta"] is not None else x.new_zeros(n), (x - mean[:, None]) * rstd[:, None],
                          s["gamma"].double())
        return y, mean if case["norm"] == "layer" else None, rstd
    if op == "norm_grad":
        # y_i = gamma_i h_i + beta_i, h = (x - mu) r; with u = gamma dy:
        # dx = r (u - h <u, h> / m - [layer] <u, 1> / m), dgamma = sum_t dy h, dbeta = sum_t dy
        x, dy, gamma, r = (s[n].double() for n in ("x", "dy", "gamma", "rstd"))
        layer = case["norm"] == "layer"
        h = x - s["mean"].double()[:, None] if layer else x
        h = h * r[:, None]
        u, m = dy * gamma, x.shape[1]
        along = torch.einsum("tm,tm->t", u, h) / m
        across = u.sum(1) / m if layer else torch.zeros_like(along)
        dx = (u - torch.einsum("t,tm->tm", along, h) - across[:, None]) * r[:, None]
        return dx, torch.einsum("tm,tm->m", dy, h), torch.einsum("tm->m", dy) if layer else None
    if op == "product":
        y = []
        ends = [0, s["rows"]] if s["offsets"] is None else s["offsets"].tolist()
        for e in range(case["E"]):
            at = torch.arange(ends[e], ends[e + 1], device="cuda")
            at = at if s["perm"] is None else s["perm"].long()[at] // case["k"]
            sums = torch.mm(s["x"][at].double(), s["w"][e].double().t())
            y.append(sums * torch.outer(s["x_scale"][at].double(), s["w_scale"][e].double()))
        return torch.cat(y)
    k = case["k"]
    a = s["perm"].long()  # the assignment of each row
    t, j = a // k, a % k
    if op == "sort":
        return s["x"].double().index_select(0, t)
    r = s["r"].double()
    if op in ("sort_grad", "combine"):
        weight = s["w"].double()[t, j] if op == "combine" else torch.ones_like(t, dtype=torch.float64)
        return r.new_zeros(case["T"], case["m"]).index_add_(0, t, r * weight[:, None])
    dy = s["x"].double()
    dw = torch.zeros(case["T"], k, dtype=torch.float64, device="cuda")
    dw[t, j] = torch.einsum("rm,rm->r", dy[t], r)
    return dy[t] * s["w"].double()[t, j][:, None], dw
