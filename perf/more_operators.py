"""The operators that make an MoE block trainable and its input servable in 8 bits, as cases
to be timed and compared.

Five kinds of call: the residual added and normalised (forward, with int8 codes and their
scales where a product in int8 follows, and backward), the experts' gated feed-forward block
on plain weights (forward, keeping what its gradient needs, and backward with the weight
gradients), and the gradient of the routing.

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


def _norm(name, op, norm, dtype, T, m, out="y"):
    return {"name": name, "op": op, "norm": norm, "dtype": dtype, "T": T, "m": m, "out": out}


def _ffn(name, op, T, k, E, m, p, dtype, save=False):
    return {"name": name, "op": op, "T": T, "k": k, "E": E, "m": m, "p": p, "dtype": dtype, "save": save}


def _route(name, T, k, E, m, dtype, aux):
    return {"name": name, "op": "route_grad", "T": T, "k": k, "E": E, "m": m, "dtype": dtype, "aux": aux}


def listed():
    return [
        # a decode step: the residual stream and the router's rows; a launch's latency is what counts
        _norm("add_norm_decode", "add_norm", "rms", "bf16", 16, 4096),
        # the prefill batch in front of an int8 product: rows for the router, codes and scales in one pass
        _norm("add_norm_prefill", "add_norm", "rms", "bf16", 8192, 4096, "both"),
        # the same batch in training: the residual stream's gradient and gamma's
        _norm("add_norm_grad_prefill", "add_norm_grad", "rms", "bf16", 8192, 4096),
        # a ragged fp32 batch with a layer norm
        _norm("add_norm_grad_ragged", "add_norm_grad", "layer", "f32", 777, 5000),
        # one token through two of the Mixtral-shaped experts: their weights stream once
        _ffn("ffn_token", "ffn", 1, 2, 8, 4096, 14336, "bf16"),
        # a decode batch over sixteen Phi-shaped experts
        _ffn("ffn_decode", "ffn", 64, 2, 16, 4096, 6400, "bf16"),
        # a training batch's forward pass, gate and up kept
        _ffn("ffn_prefill", "ffn", 8192, 2, 8, 4096, 14336, "bf16", True),
        # a ragged fp32 batch, sizes that no tile divides
        _ffn("ffn_ragged", "ffn", 333, 3, 12, 1000, 1720, "f32", True),
        # a training batch's backward pass over sixteen experts, all weight gradients
        _ffn("ffn_grad_train", "ffn_grad", 8192, 2, 16, 4096, 6400, "bf16"),
        # the same ragged, in fp32
        _ffn("ffn_grad_ragged", "ffn_grad", 517, 2, 5, 1000, 712, "f32"),
        # the routing's gradient over a training batch, joined with the experts' part
        _route("route_grad_train", 8192, 2, 8, 4096, "bf16", False),
        # ragged, many experts, with a loss on the logits themselves (a load-balancing term)
        _route("route_grad_ragged", 1237, 4, 33, 1000, "f32", True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["add_norm", "add_norm", "add_norm_grad", "ffn", "ffn", "ffn_grad", "ffn_grad", "route_grad"])
    dtype = rng.choice(["bf16", "f32"])
    if op in ("add_norm", "add_norm_grad"):
        m = _log(rng, 64, 16384, 8)
        return {"op": op, "norm": rng.choice(["layer", "rms"]), "dtype": dtype,
                "T": _log(rng, 1, min(16384, (1 << 24) // m)), "m": m,
                "out": rng.choice(["y", "codes", "both"]) if op == "add_norm" else "y"}
    E = rng.choice([1, 2, 5, 8, 16, 33, 64])
    k = min(E, rng.choice([1, 2, 2, 3, 4, 8]))
    if op == "route_grad":
        m = _log(rng, 64, 8192, 8)
        return {"op": op, "T": _log(rng, 1, min(8192, (1 << 25) // m)), "k": k, "E": E, "m": m, "dtype": dtype,
                "aux": rng.choice([True, False])}
    m, p = _log(rng, 64, 8192, 8), _log(rng, 64, 14336, 8)
    while E * m * p > 1 << 29:
        E = (E + 1) // 2
    k = min(E, k)
    k = rng.choice([0, k]) if E == 1 else k  # 0: dense, without a dispatch
    most = min(16384, (1 << (37 if dtype == "bf16" else 34)) // (m * p))
    return {"op": op, "T": max(1, _log(rng, 1, most) // max(1, k)), "k": k, "E": E, "m": m, "p": p, "dtype": dtype,
            "save": rng.choice([True, False]) if op == "ffn" else False}


def work(case):
    op, T, m, s = case["op"], case["T"], case["m"], SIZE[case["dtype"]]
    if op in ("add_norm", "add_norm_grad"):
        wide = 1 if case["norm"] == "rms" else 2  # gamma (and beta); rstd (and mean)
        if op == "add_norm_grad":
            return {"bytes": 4 * T * m * s + 4 * m + 4 * wide * (m + T), "flops": 17 * T * m}
        out = (s if case["out"] != "codes" else 0) * T * m + ((m + 4) * T if case["out"] != "y" else 0)
        return {"bytes": 3 * T * m * s + out + 4 * wide * (m + T), "flops": 10 * T * m}
    k, E = case["k"], case["E"]
    if op == "route_grad":
        return {"bytes": 3 * T * m * s + 8 * m * E + 12 * T * k + 4 * T * E * (2 if case["aux"] else 1) + 4 * E,
                "flops": 4 * T * m * (E if case["aux"] else k)}
    R, p = T * max(1, k), case["p"]
    index = 4 * (E + 1) + 4 * R if k else 0
    weights = 3 * min(E, R) * m * p * s
    if op == "ffn":
        return {"bytes": T * m * s + weights + R * m * s + (2 * R * p * s if case["save"] else 0) + index,
                "flops": 6 * R * m * p}
    return {"bytes": T * m * s + 2 * R * m * s + 2 * R * p * s + weights + 3 * E * m * p * s + index,
            "flops": 12 * R * m * p}


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


def _weights(g, E, rows, cols, dtype):
    """E matrices of a layer's usual scale: unit rows in, unit rows out."""
    return torch.randn(E, rows, cols, generator=g, device="cuda").mul_(rows ** -0.5).to(DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, T, m, dt = case["op"], case["T"], case["m"], DTYPES[case["dtype"]]
    s = {"case": case, "op": op}
    if op in ("add_norm", "add_norm_grad"):
        layer = case["norm"] == "layer"
        s["x"] = torch.randn(T, m, generator=g, device="cuda").mul_(0.5).to(dt)  # a block's output
        s["residual"] = _activations(g, T, m, case["dtype"])
        s["gamma"] = 1 + 0.2 * torch.randn(m, generator=g, device="cuda")
        s["beta"] = 0.1 * torch.randn(m, generator=g, device="cuda") if layer else None
        if op == "add_norm":
            s["sum"] = torch.empty_like(s["x"])
            s["y"] = torch.empty_like(s["x"]) if case["out"] != "codes" else None
            s["codes"] = torch.empty(T, m, dtype=torch.int8, device="cuda") if case["out"] != "y" else None
            s["scale"] = torch.empty(T, device="cuda") if case["out"] != "y" else None
            s["mean"] = torch.empty(T, device="cuda") if layer else None
            s["rstd"] = torch.empty(T, device="cuda")
            return s
        # what the forward pass left
        h = s.pop("x").double() + s.pop("residual").double()
        mean = h.mean(1) if layer else torch.zeros(T, dtype=torch.float64, device="cuda")
        s["rstd"] = ((h - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        s["mean"] = mean.float() if layer else None
        s["sum"] = h.to(dt)
        s["dy"] = torch.randn(T, m, generator=g, device="cuda").to(dt)
        s["dsum"] = torch.randn(T, m, generator=g, device="cuda").to(dt)
        s["dx"] = torch.empty_like(s["sum"])
        s["dgamma"] = torch.empty(m, device="cuda")
        s["dbeta"] = torch.empty(m, device="cuda") if layer else None
        if own:
            import mixture_experts_layer_gemv_amd as M

            s["bytes"] = M.moe_norm_backward_workspace_size(T, m)
            s["workspace"] = torch.empty(max(256, s["bytes"]), dtype=torch.uint8, device="cuda")
        return s
    k, E = case["k"], case["E"]
    s["x"] = _activations(g, T, m, case["dtype"])
    if op == "route_grad":
        s["idx"] = _choices(g, T, k, E).to(torch.int32)
        s["w"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
        s["dw"] = torch.randn(T, k, generator=g, device="cuda")
        s["dl_add"] = 0.01 * torch.randn(T, E, generator=g, device="cuda") if case["aux"] else None
        s["wr"] = torch.randn(m, E, generator=g, device="cuda").mul_(m ** -0.5)
        s["dx_add"] = torch.randn(T, m, generator=g, device="cuda").to(dt)
        s["dl"] = torch.empty(T, E, device="cuda")
        s["dx"] = torch.empty_like(s["x"])
        s["dwr"] = torch.empty(m, E, device="cuda")
        s["db"] = torch.empty(E, device="cuda")
        if own:
            import mixture_experts_layer_gemv_amd as M

            s["bytes"] = M.moe_route_backward_workspace_size(T, m, E)
            s["workspace"] = torch.empty(max(256, s["bytes"]), dtype=torch.uint8, device="cuda")
        return s
    p = case["p"]
    s["wg"], s["wu"] = _weights(g, E, m, p, case["dtype"]), _weights(g, E, m, p, case["dtype"])
    s["wd"] = _weights(g, E, p, m, case["dtype"])
    s["rows"] = s["most"] = R = T * max(1, k)
    s["offsets"] = s["perm"] = None
    if k:
        idx = _choices(g, T, k, E).reshape(-1)
        s["perm"] = torch.sort(idx, stable=True).indices.to(torch.int32)
        counts = torch.bincount(idx, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())  # rows that the fullest expert takes
    s["gate"] = s["up"] = None
    if op == "ffn_grad":
        # as the forward pass leaves them: of the rows' scale
        s["gate"] = torch.randn(R, p, generator=g, device="cuda").mul_(1.2).to(dt)
        s["up"] = torch.randn(R, p, generator=g, device="cuda").mul_(1.2).to(dt)
        s["dy"] = torch.randn(R, m, generator=g, device="cuda").to(dt)
        s["dx"] = torch.empty(R, m, dtype=dt, device="cuda")
        s["dwg"], s["dwu"], s["dwd"] = (torch.empty_like(s[n]) for n in ("wg", "wu", "wd"))
    else:
        s["y"] = torch.empty(R, m, dtype=dt, device="cuda")
        if case["save"]:
            s["gate"], s["up"] = (torch.empty(R, p, dtype=dt, device="cuda") for _ in range(2))
    if own:
        import mixture_experts_layer_gemv_amd as M

        code = M.MOE_BF16 if dt == torch.bfloat16 else M.MOE_F32
        s["bytes"] = M.moe_gated_ffn_workspace_size(code, R, m, p, E, 1 if op == "ffn_grad" else 0)
        s["workspace"] = torch.empty(max(256, s["bytes"]), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ---------------------------------------------------------------------


def run(s):
    if own:
        return _own(s)
    return {"add_norm": _plain_add_norm, "add_norm_grad": _plain_add_norm_grad, "ffn": _plain_ffn,
            "ffn_grad": _plain_ffn_grad, "route_grad": _plain_route_grad}[s["op"]](s)


def _values(codes, scale):
    """What codes stand for: seven bits times a power of two, which bf16 holds exactly."""
    return codes * scale.to(torch.bfloat16)[:, None]


def _scales(y):
    """2^X, X the smallest integer with max|y| <= 127 * 2^X (0 where a row is all zeros)."""
    top = y.abs().amax(1).double() / 127
    fraction, exponent = torch.frexp(top)
    exponent = torch.where(fraction == 0.5, exponent - 1, exponent)
    return torch.ldexp(torch.ones_like(top), torch.where(top > 0, exponent, 0)).float()


def _plain_add_norm(s):
    h = s["x"].float() + s["residual"].float()
    mean = h.mean(1) if s["case"]["norm"] == "layer" else None
    d = h - mean[:, None] if mean is not None else h
    rstd = (d.square().mean(1) + EPS).rsqrt()
    y = d * rstd[:, None] * s["gamma"]
    if s["beta"] is not None:
        y = y + s["beta"]
    out = {"sum": h.to(s["x"].dtype), "rstd": rstd}
    if mean is not None:
        out["mean"] = mean
    if s["case"]["out"] != "codes":
        out["y"] = y.to(s["x"].dtype)
    if s["case"]["out"] != "y":
        out["scale"] = _scales(y)
        out["values"] = _values(torch.round(y / out["scale"][:, None]).to(torch.int8), out["scale"])
    return out


def _plain_add_norm_grad(s):
    h, dy = s["sum"].float(), s["dy"].float()
    hat = (h - s["mean"][:, None] if s["mean"] is not None else h) * s["rstd"][:, None]
    g = dy * s["gamma"]
    dx = g - hat * (g * hat).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - g.mean(1, keepdim=True)
    dx = s["dsum"].float() + dx * s["rstd"][:, None]
    return dx.to(s["sum"].dtype), (dy * hat).sum(0), dy.sum(0) if s["mean"] is not None else None


def _by_expert(s):
    """Each row's token, expert and place among its expert's rows."""
    c, at = s["case"], torch.arange(s["rows"], device="cuda")
    if s["perm"] is None:
        return at, torch.zeros_like(at), at
    expert = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    return (s["perm"] // c["k"]).long(), expert, at - s["offsets"].long()[expert]


def _padded(s, rows, expert, place):
    """Rows [E][most][columns] in 32 bits, zeros past an expert's last."""
    out = torch.zeros(s["case"]["E"], s["most"], rows.shape[1], device="cuda")
    out[expert, place] = rows.float()
    return out


def _plain_ffn(s):
    token, expert, place = _by_expert(s)
    dt = s["x"].dtype
    x = _padded(s, s["x"][token], expert, place)
    gate, up = torch.bmm(x, s["wg"].float()), torch.bmm(x, s["wu"].float())
    y = torch.bmm(gate * torch.sigmoid(gate) * up, s["wd"].float())[expert, place].to(dt)
    if not s["case"]["save"]:
        return y
    return y, gate[expert, place].to(dt), up[expert, place].to(dt)


def _plain_ffn_grad(s):
    token, expert, place = _by_expert(s)
    dt = s["x"].dtype
    x, dy, gate, up = (_padded(s, r, expert, place) for r in (s["x"][token], s["dy"], s["gate"], s["up"]))
    sg = torch.sigmoid(gate)
    h = gate * sg * up
    dh = torch.bmm(dy, s["wd"].float().transpose(1, 2).contiguous())
    dwd = torch.bmm(h.transpose(1, 2).contiguous(), dy).to(dt)
    dgate, dup = dh * up * sg * (1 + gate * (1 - sg)), dh * gate * sg
    xt = x.transpose(1, 2).contiguous()
    dwg, dwu = torch.bmm(xt, dgate).to(dt), torch.bmm(xt, dup).to(dt)
    dx = torch.bmm(dgate, s["wg"].float().transpose(1, 2).contiguous())
    dx = dx + torch.bmm(dup, s["wu"].float().transpose(1, 2).contiguous())
    return dx[expert, place].to(dt), dwg, dwu, dwd


def _plain_route_grad(s):
    w, dw = s["w"], s["dw"]
    each = w * (dw - (w * dw).sum(1, keepdim=True))
    hit = s["idx"][:, :, None] == torch.arange(s["case"]["E"], device="cuda")
    dl = (hit * each[:, :, None]).sum(1)
    if s["dl_add"] is not None:
        dl = dl + s["dl_add"]
    dx = s["dx_add"].float() + dl @ s["wr"].t()
    return dl, dx.to(s["x"].dtype), s["x"].float().t() @ dl, dl.sum(0)


def _own(s):
    import mixture_experts_layer_gemv_amd as M

    c, op = s["case"], s["op"]
    T, m = c["T"], c["m"]
    dt = M.MOE_BF16 if c["dtype"] == "bf16" else M.MOE_F32
    if op in ("add_norm", "add_norm_grad"):
        kind = M.MOE_NORM_LAYER if c["norm"] == "layer" else M.MOE_NORM_RMS
        if op == "add_norm_grad":
            M.moe_add_norm_backward(s["dy"], s["dsum"], s["sum"], dt, kind, s["gamma"], s["mean"], s["rstd"], T, m,
                                    s["dx"], s["dgamma"], s["dbeta"], s["workspace"], s["bytes"])
            return s["dx"], s["dgamma"], s["dbeta"]
        M.moe_add_norm_forward(s["x"], s["residual"], dt, kind, s["gamma"], s["beta"], EPS, T, m, s["sum"], s["y"],
                               s["codes"], s["scale"], s["mean"], s["rstd"])
        out = {n: s[n] for n in ("sum", "rstd", "mean", "y", "scale") if s[n] is not None}
        if s["codes"] is not None:
            out["values"] = _values(s["codes"], s["scale"])
        return out
    if op == "route_grad":
        M.moe_route_backward(s["dw"], s["idx"], s["w"], s["dl_add"], s["x"], dt, s["wr"], s["dx_add"], T, m, c["E"],
                             c["k"], s["dl"], s["dx"], s["dwr"], s["db"], s["workspace"], s["bytes"])
        return s["dl"], s["dx"], s["dwr"], s["db"]
    where = (s["offsets"], s["perm"], T, max(1, c["k"]), s["rows"], m, c["p"], c["E"])
    if op == "ffn":
        M.moe_gated_ffn_forward(s["x"], dt, s["wg"], s["wu"], s["wd"], *where, s["y"], s["gate"], s["up"],
                                s["workspace"], s["bytes"])
        return (s["y"], s["gate"], s["up"]) if c["save"] else s["y"]
    M.moe_gated_ffn_backward(s["dy"], s["x"], dt, s["wg"], s["wu"], s["wd"], s["gate"], s["up"], *where, s["dx"],
                             s["dwg"], s["dwu"], s["dwd"], s["workspace"], s["bytes"])
    return s["dx"], s["dwg"], s["dwu"], s["dwd"]


# ---- the definitions in 64 bits -----------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "add_norm":
        h = s["x"].double() + s["residual"].double()
        n = h.shape[1]
        layer = case["norm"] == "layer"
        mean = h.sum(1) / n if layer else h.new_zeros(len(h))
        d = h - mean[:, None]
        rstd = 1 / torch.sqrt(torch.einsum("tm,tm->t", d, d) / n + EPS)
        y = torch.addcmul(s["beta"].double() if layer else h.new_zeros(n), d * rstd[:, None], s["gamma"].double())
        out = {"sum": h, "rstd": rstd}
        if layer:
            out["mean"] = mean
        if case["out"] != "codes":
            out["y"] = y
        if case["out"] != "y":
            # the smallest power of two that 127 steps of reach the row's largest magnitude
            out["scale"] = torch.exp2(torch.ceil(torch.log2(y.abs().amax(1).clamp_min(1e-300) / 127)))
            out["values"] = torch.round(y / out["scale"][:, None]) * out["scale"][:, None]
        return out
    if op == "add_norm_grad":
        # y_i = gamma_i h_i + beta_i, h = (s - mu) r; with u = gamma dy:
        # ds = dsum + r (u - h <u, h> / m - [layer] <u, 1> / m), dgamma = sum_t dy h, dbeta = sum_t dy
        x, dy, gamma, r = (s[n].double() for n in ("sum", "dy", "gamma", "rstd"))
        layer = case["norm"] == "layer"
        h = (x - s["mean"].double()[:, None] if layer else x) * r[:, None]
        u, m = dy * gamma, x.shape[1]
        along = torch.einsum("tm,tm->t", u, h) / m
        across = u.sum(1) / m if layer else torch.zeros_like(along)
        dx = torch.addcmul(s["dsum"].double(), u - torch.einsum("t,tm->tm", along, h) - across[:, None], r[:, None])
        return dx, torch.einsum("tm,tm->m", dy, h), torch.einsum("tm->m", dy) if layer else None
    if op == "route_grad":
        # w = softmax of the chosen logits: dl_j = w_j dw_j - w_j <w, dw>
        w, dw = s["w"].double(), s["dw"].double()
        mine = torch.addcmul(w * dw, w, -torch.einsum("tk,tk->t", w, dw)[:, None])
        dl = torch.zeros(case["T"], case["E"], dtype=torch.float64, device="cuda")
        dl.scatter_(1, s["idx"].long(), mine)
        if case["aux"]:
            dl += s["dl_add"]
        dx = torch.addmm(s["dx_add"].double(), dl, s["wr"].double().t())
        return dl, dx, torch.mm(s["x"].double().t(), dl), torch.einsum("te->e", dl)
    ends = [0, s["rows"]] if s["offsets"] is None else s["offsets"].tolist()
    parts = []
    for e in range(case["E"]):
        at = torch.arange(ends[e], ends[e + 1], device="cuda")
        x = s["x"][at if s["perm"] is None else s["perm"].long()[at] // case["k"]].double()
        wg, wu, wd = (s[n][e].double() for n in ("wg", "wu", "wd"))
        if op == "ffn":
            g, u = torch.mm(x, wg), torch.mm(x, wu)
            parts.append((torch.mm(g / (1 + torch.exp(-g)) * u, wd), g, u))
            continue
        g, u, dy = (s[n][at].double() for n in ("gate", "up", "dy"))
        sg = 1 / (1 + torch.exp(-g))
        silu = g * sg
        dh = torch.mm(dy, wd.t())
        dg, du = dh * u * (sg + silu * (1 - sg)), dh * silu
        parts.append((torch.addmm(torch.mm(dg, wg.t()), du, wu.t()), torch.mm(x.t(), dg)[None], torch.mm(x.t(), du)[None],
                      torch.mm((silu * u).t(), dy)[None]))
    out = tuple(torch.cat(p) for p in zip(*parts))
    return out[0] if op == "ffn" and not case["save"] else out
