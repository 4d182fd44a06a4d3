"""The trainable block's operators (residual norm, gated feed-forward, routing
gradient) refuse bad arguments before anything is launched, without a GPU."""
import ctypes

import pytest

FAKE = 0x7F0000000000  # never dereferenced: every call below fails validation or has nothing to do
Z = None


@pytest.fixture(scope="module")
def M():
    import mixture_experts_layer_gemv_amd as m

    m.lib()
    return m


def _refused(M, fn, want, *args):
    rc = getattr(M.lib(), fn)(*args)
    assert rc == want, (fn, args, rc, M.moe_last_error())
    assert (M.moe_last_error() == "") == (want == M.MOE_OK)


def test_add_norm_forward(M):
    bad, uns = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED

    def call(want, x=FAKE, r=FAKE, dt=1, norm=1, g=FAKE, b=FAKE, eps=1e-5, T=4, m=64, s=FAKE, y=FAKE + 4096, c=FAKE,
             sc=FAKE, mean=FAKE, rstd=FAKE):
        _refused(M, "moe_add_norm_forward", want, x, r, dt, norm, g, b, eps, T, m, s, y, c, sc, mean, rstd, Z)

    for a in [dict(x=Z), dict(g=Z), dict(y=Z, c=Z, sc=Z), dict(c=Z), dict(sc=Z), dict(y=FAKE), dict(x=FAKE + 8), dict(r=FAKE + 2),
              dict(s=FAKE + 8), dict(y=FAKE + 8), dict(c=FAKE + 8), dict(g=FAKE + 4), dict(b=FAKE + 4), dict(T=-1), dict(m=0),
              dict(m=-8), dict(norm=0), dict(norm=3), dict(eps=-1.0), dict(eps=2.0), dict(eps=float("nan")), dict(norm=2),
              dict(norm=2, b=Z), dict(norm=2, mean=Z)]:
        call(bad, **a)
    for a in [dict(m=12), dict(m=16392), dict(dt=2), dict(dt=-1)]:
        call(uns, **a)
    call(M.MOE_OK, T=0)
    call(M.MOE_OK, T=0, x=Z, y=Z, g=Z, c=Z, sc=Z)


def test_add_norm_backward(M):
    bad, uns = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED
    need = M.moe_norm_backward_workspace_size(4, 64)

    def call(want, dy=FAKE, ds=FAKE, s=FAKE, dt=1, norm=1, g=FAKE, mean=FAKE, rstd=FAKE, T=4, m=64, dx=FAKE, dg=FAKE,
             db=FAKE, ws=FAKE, n=need):
        _refused(M, "moe_add_norm_backward", want, dy, ds, s, dt, norm, g, mean, rstd, T, m, dx, dg, db, ws, n, Z)

    for a in [dict(dy=Z), dict(s=Z), dict(g=Z), dict(rstd=Z), dict(mean=Z), dict(dx=Z, dg=Z, db=Z), dict(dx=FAKE + 8),
              dict(ds=FAKE + 8), dict(dg=FAKE + 4), dict(dy=FAKE + 2), dict(s=FAKE + 2), dict(g=FAKE + 4), dict(norm=2),
              dict(norm=2, mean=Z), dict(norm=2, db=Z), dict(norm=0), dict(T=-1), dict(m=0), dict(ws=FAKE + 16)]:
        call(bad, **a)
    for a in [dict(m=20), dict(m=32768), dict(dt=4)]:
        call(uns, **a)
    for a in [dict(ws=Z), dict(n=need - 1), dict(n=0)]:
        call(M.MOE_ERR_WORKSPACE, **a)
    call(M.MOE_OK, T=0, dg=Z, db=Z)


BAD = [dict(T=-1), dict(rows=-1), dict(m=0), dict(p=0), dict(E=0), dict(topk=0), dict(off=Z), dict(perm=Z), dict(T=0),
       dict(x=FAKE + 8), dict(wg=Z), dict(wu=Z), dict(wd=Z), dict(wg=FAKE + 8), dict(wu=FAKE + 2), dict(wd=FAKE + 8),
       dict(ws=FAKE + 16)]
UNSUPPORTED = [dict(dt=2), dict(dt=-1), dict(m=12), dict(p=100), dict(E=65), dict(m=(1 << 20) + 8), dict(p=1 << 21),
               dict(rows=1 << 30, m=1 << 15), dict(E=64, m=1 << 20, p=1 << 20)]


def test_gated_forward(M):
    need = M.moe_gated_ffn_workspace_size(M.MOE_BF16, 8, 64, 72, 4, 0)

    def call(want, x=FAKE, dt=1, wg=FAKE, wu=FAKE, wd=FAKE, off=FAKE, perm=FAKE, T=4, topk=2, rows=8, m=64, p=72, E=4,
             y=FAKE, g=FAKE, u=FAKE, ws=FAKE, n=need):
        _refused(M, "moe_gated_ffn_forward", want, x, dt, wg, wu, wd, off, perm, T, topk, rows, m, p, E, y, g, u, ws, n, Z)

    for a in BAD + [dict(x=Z), dict(y=Z), dict(y=FAKE + 8), dict(g=Z), dict(u=Z), dict(g=FAKE + 8), dict(u=FAKE + 8)]:
        call(M.MOE_ERR_INVALID_ARG, **a)
    for a in UNSUPPORTED:
        call(M.MOE_ERR_UNSUPPORTED, **a)
    for a in [dict(ws=Z), dict(n=need - 1)]:
        call(M.MOE_ERR_WORKSPACE, **a)
    call(M.MOE_OK, rows=0)
    call(M.MOE_OK, rows=0, T=0, perm=Z, off=Z, E=1, x=Z, y=Z, ws=Z, n=0, wg=Z, wu=Z, wd=Z, g=Z, u=Z)


def test_gated_backward(M):
    need = M.moe_gated_ffn_workspace_size(M.MOE_F32, 8, 64, 72, 4, 1)

    def call(want, dy=FAKE, x=FAKE, dt=0, wg=FAKE, wu=FAKE, wd=FAKE, g=FAKE, u=FAKE, off=FAKE, perm=FAKE, T=4, topk=2,
             rows=8, m=64, p=72, E=4, dx=FAKE, dwg=FAKE, dwu=FAKE, dwd=FAKE, ws=FAKE, n=need):
        _refused(M, "moe_gated_ffn_backward", want, dy, x, dt, wg, wu, wd, g, u, off, perm, T, topk, rows, m, p, E, dx, dwg,
                 dwu, dwd, ws, n, Z)

    none = dict(dx=Z, dwg=Z, dwu=Z, dwd=Z)
    for a in BAD + [dict(dy=Z), dict(x=Z), dict(g=Z), dict(u=Z), none, dict(dwg=Z), dict(dwu=Z), dict(dy=FAKE + 4),
                    dict(dx=FAKE + 8), dict(dwg=FAKE + 8), dict(dwd=FAKE + 4), dict(g=FAKE + 4)]:
        call(M.MOE_ERR_INVALID_ARG, **a)
    for a in UNSUPPORTED:
        call(M.MOE_ERR_UNSUPPORTED, **a)
    for a in [dict(ws=Z), dict(n=need - 1)]:
        call(M.MOE_ERR_WORKSPACE, **a)
    call(M.MOE_OK, rows=0, dwg=Z, dwu=Z, dwd=Z)


def test_gated_workspace_size(M):
    size = M.moe_gated_ffn_workspace_size
    assert size(M.MOE_BF16, 0, 64, 64, 1, 0) == 0
    assert size(M.MOE_BF16, 1000, 64, 72, 8, 0) >= 1000 * 72 * 2
    assert size(M.MOE_F32, 1000, 64, 72, 8, 1) >= 1000 * (3 * 72 + 64) * 4
    L, n = M.lib(), ctypes.c_size_t()
    assert L.moe_gated_ffn_workspace_size(1, 8, 64, 64, 4, 0, Z) == M.MOE_ERR_INVALID_ARG
    assert L.moe_gated_ffn_workspace_size(1, -1, 64, 64, 4, 0, ctypes.byref(n)) == M.MOE_ERR_INVALID_ARG
    for a in [(3, 8, 64, 64, 4, 0), (1, 8, 60, 64, 4, 0), (1, 8, 64, 60, 4, 1), (1, 8, 64, 64, 65, 0)]:
        assert L.moe_gated_ffn_workspace_size(*a, ctypes.byref(n)) == M.MOE_ERR_UNSUPPORTED, a


def test_route_backward(M):
    bad, uns = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED
    need = M.moe_route_backward_workspace_size(4, 64, 8)

    def call(want, dw=FAKE, idx=FAKE, w=FAKE, dla=FAKE, x=FAKE, dt=1, wr=FAKE, dxa=FAKE, T=4, m=64, E=8, k=2, dl=FAKE,
             dx=FAKE, dwr=FAKE, db=FAKE, ws=FAKE, n=need):
        _refused(M, "moe_route_backward", want, dw, idx, w, dla, x, dt, wr, dxa, T, m, E, k, dl, dx, dwr, db, ws, n, Z)

    for a in [dict(dw=Z), dict(idx=Z), dict(w=Z), dict(x=Z), dict(wr=Z), dict(dl=Z), dict(T=-1), dict(m=0), dict(E=0),
              dict(k=0), dict(k=9), dict(x=FAKE + 8), dict(dxa=FAKE + 8), dict(dx=FAKE + 8), dict(ws=FAKE + 16)]:
        call(bad, **a)
    for a in [dict(m=12), dict(E=65), dict(dt=2), dict(m=(1 << 20) + 8), dict(T=1 << 30, k=4), dict(T=(1 << 30) + 1, k=1)]:
        call(uns, **a)
    for a in [dict(ws=Z), dict(n=need - 1)]:
        call(M.MOE_ERR_WORKSPACE, **a)
    call(M.MOE_OK, T=0, dwr=Z, db=Z)
    size = M.moe_route_backward_workspace_size
    assert size(0, 64, 8) == 0 and size(1, 64, 8) > 0
    assert size(1 << 20, 4096, 8) == size(1 << 22, 4096, 8)  # bounded by the launch, not by T
    with pytest.raises(M.MoeError):
        size(4, 60, 8)


def test_route_backward_outputs_over_inputs(M):
    """Rows that several workgroups read while one writes them: every other argument is as it should be."""
    dw, idx, w, dla, x, wr, dxa, dl, dx, dwr, db, ws = (ctypes.c_void_p(FAKE + (i << 20)) for i in range(12))
    n = M.moe_route_backward_workspace_size(4, 64, 8)
    for over in (dla, dw, w):
        _refused(M, "moe_route_backward", M.MOE_ERR_INVALID_ARG, dw, idx, w, dla, x, 1, wr, dxa, 4, 64, 8, 2, over, dx, dwr, db,
                 ws, n, Z)
    _refused(M, "moe_route_backward", M.MOE_ERR_INVALID_ARG, dw, idx, w, dla, x, 1, wr, dxa, 4, 64, 8, 2, dl, x, dwr, db, ws, n, Z)


def test_binding_refuses_host_tensors(M):
    import torch

    x, g = torch.zeros(4, 64), torch.ones(64)
    calls = [lambda: M.moe_add_norm_forward(x, x, M.MOE_F32, M.MOE_NORM_RMS, g, None, 1e-5, 4, 64, None, x, stream=0),
             lambda: M.moe_add_norm_backward(x, x, x, M.MOE_F32, M.MOE_NORM_RMS, g, None, g, 4, 64, x, None, None, stream=0),
             lambda: M.moe_gated_ffn_forward(x, M.MOE_F32, x, x, x, None, None, 4, 1, 4, 64, 64, 1, x, stream=0),
             lambda: M.moe_gated_ffn_backward(x, x, M.MOE_F32, x, x, x, x, x, None, None, 4, 1, 4, 64, 64, 1, x, None, None,
                                              None, stream=0),
             lambda: M.moe_route_backward(x, x, x, None, x, M.MOE_F32, x, None, 4, 64, 8, 2, x, stream=0)]
    for call in calls:
        with pytest.raises(M.MoeError) as ei:
            call()
        assert ei.value.status == M.MOE_ERR_INVALID_ARG and "GPU" in ei.value.message
