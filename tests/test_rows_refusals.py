"""The row operators (norm, permute, combine, int8 product) refuse bad
arguments before anything is launched, without a GPU."""
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


def test_norm_forward(M):
    bad, uns = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED

    def call(want, x=FAKE, dt=1, norm=1, g=FAKE, b=FAKE, eps=1e-5, T=4, m=64, y=FAKE, mean=FAKE, rstd=FAKE):
        _refused(M, "moe_norm_forward", want, x, dt, norm, g, b, eps, T, m, y, mean, rstd, Z)

    for a in [dict(x=Z), dict(g=Z), dict(y=Z), dict(x=FAKE + 8), dict(y=FAKE + 2), dict(g=FAKE + 4), dict(b=FAKE + 4),
              dict(T=-1), dict(m=0), dict(m=-8), dict(norm=0), dict(norm=3), dict(eps=-1.0), dict(eps=2.0),
              dict(eps=float("nan")), dict(norm=2), dict(norm=2, b=Z), dict(norm=2, mean=Z)]:
        call(bad, **a)
    for a in [dict(m=12), dict(m=16392), dict(dt=2), dict(dt=-1)]:
        call(uns, **a)
    call(M.MOE_OK, T=0)
    call(M.MOE_OK, T=0, x=Z, y=Z, g=Z)


def test_norm_backward(M):
    bad, uns = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED
    need = M.moe_norm_backward_workspace_size(4, 64)
    assert need >= 2 * 4 * 64

    def call(want, dy=FAKE, x=FAKE, dt=1, norm=1, g=FAKE, mean=FAKE, rstd=FAKE, T=4, m=64, dx=FAKE, dg=FAKE, db=FAKE,
             ws=FAKE, n=need):
        _refused(M, "moe_norm_backward", want, dy, x, dt, norm, g, mean, rstd, T, m, dx, dg, db, ws, n, Z)

    for a in [dict(dy=Z), dict(x=Z), dict(g=Z), dict(rstd=Z), dict(mean=Z), dict(dx=Z, dg=Z, db=Z), dict(dx=FAKE + 8),
              dict(dg=FAKE + 4), dict(db=FAKE + 8), dict(dy=FAKE + 2), dict(x=FAKE + 2), dict(g=FAKE + 4),
              dict(norm=2), dict(norm=2, mean=Z), dict(norm=2, db=Z), dict(norm=0), dict(T=-1), dict(m=0),
              dict(ws=FAKE + 16)]:
        call(bad, **a)
    for a in [dict(m=20), dict(m=32768), dict(dt=4)]:
        call(uns, **a)
    for a in [dict(ws=Z), dict(n=need - 1), dict(n=0)]:
        call(M.MOE_ERR_WORKSPACE, **a)
    call(M.MOE_OK, T=0, dg=Z, db=Z)


def test_norm_workspace_size(M):
    size = M.moe_norm_backward_workspace_size
    assert size(0, 64) == 0
    assert size(1, 64) == 2 * 64 * 4
    assert size(1 << 20, 4096) == size(1 << 21, 4096)  # bounded by the launch, not by T
    n = ctypes.c_size_t()
    L = M.lib()
    assert L.moe_norm_backward_workspace_size(4, 64, Z) == M.MOE_ERR_INVALID_ARG
    assert L.moe_norm_backward_workspace_size(-1, 64, ctypes.byref(n)) == M.MOE_ERR_INVALID_ARG
    assert L.moe_norm_backward_workspace_size(4, 63, ctypes.byref(n)) == M.MOE_ERR_UNSUPPORTED
    with pytest.raises(M.MoeError):
        size(4, 1 << 20)


@pytest.mark.parametrize("fn", ["moe_permute_rows", "moe_permute_rows_backward", "moe_combine_rows",
                                "moe_combine_rows_backward"])
def test_assignment_operators(M, fn):
    bad, uns = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED

    def call(want, src=FAKE, dt=1, inv=FAKE, w=FAKE, T=4, m=64, k=2, rows=8, dst=FAKE, dt2=1, r=FAKE, dw=FAKE):
        if fn == "moe_permute_rows":
            args = (src, dt, inv, T, m, k, rows, dst)
        elif fn == "moe_permute_rows_backward":
            args = (src, dt, inv, T, m, k, rows, dst, dt2)
        elif fn == "moe_combine_rows":
            args = (src, dt, inv, w, T, m, k, rows, dst, dt2)
        else:
            args = (src, dt, r, dt2, inv, w, T, m, k, rows, dst, dw)
        _refused(M, fn, want, *args, Z)

    for a in [dict(src=Z), dict(inv=Z), dict(src=FAKE + 8), dict(dst=FAKE + 4), dict(T=-1), dict(m=0), dict(k=0),
              dict(rows=-1)]:
        call(bad, **a)
    for a in [dict(m=4), dict(k=65), dict(dt=3), dict(T=1 << 30, k=2)]:
        call(uns, **a)
    call(M.MOE_OK, T=0)
    if fn != "moe_permute_rows":
        call(uns, dt2=3)
    if fn == "moe_permute_rows":
        call(bad, dst=Z)
        call(M.MOE_OK, rows=0, dst=Z)
    if fn == "moe_combine_rows":
        call(bad, w=Z)
        call(bad, dst=Z)
    if fn == "moe_combine_rows_backward":
        call(bad, w=Z)
        call(bad, r=Z)
        call(bad, dst=Z, dw=Z)
        call(bad, r=FAKE + 8)


def test_quantize_codes(M):
    L = M.lib()
    assert L.moe_quantize_codes_i8(FAKE, 4, 96, FAKE, FAKE, Z) == M.MOE_ERR_UNSUPPORTED
    assert L.moe_quantize_codes_i8(FAKE, 1 << 24, 64, FAKE, FAKE, Z) == M.MOE_ERR_UNSUPPORTED
    for a in [(Z, 4, 64, FAKE, FAKE), (FAKE, 4, 64, Z, FAKE), (FAKE, 4, 64, FAKE, Z), (FAKE + 8, 4, 64, FAKE, FAKE),
              (FAKE, 4, 64, FAKE + 8, FAKE), (FAKE, -1, 64, FAKE, FAKE), (FAKE, 4, 0, FAKE, FAKE)]:
        assert L.moe_quantize_codes_i8(*a, Z) == M.MOE_ERR_INVALID_ARG, a
    assert L.moe_quantize_codes_i8(Z, 0, 64, Z, Z, Z) == M.MOE_OK


def test_matmul_i8(M):
    bad, uns = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED

    def call(want, x=FAKE, sx=FAKE, w=FAKE, sw=FAKE, off=FAKE, perm=FAKE, T=4, topk=2, rows=8, K=64, N=64, E=8, y=FAKE,
             dt=1):
        _refused(M, "moe_matmul_i8", want, x, sx, w, sw, off, perm, T, topk, rows, K, N, E, y, dt, Z)

    for a in [dict(x=Z), dict(sx=Z), dict(w=Z), dict(sw=Z), dict(y=Z), dict(x=FAKE + 8), dict(w=FAKE + 8),
              dict(sw=FAKE + 4), dict(y=FAKE + 8), dict(T=-1), dict(rows=-1), dict(K=0), dict(N=0), dict(E=0),
              dict(topk=0), dict(perm=Z), dict(off=Z), dict(T=0)]:
        call(bad, **a)
    for a in [dict(K=72), dict(N=68), dict(K=131072), dict(E=65), dict(dt=2), dict(rows=1 << 30, N=1 << 20)]:
        call(uns, **a)
    call(M.MOE_OK, rows=0)
    call(M.MOE_OK, rows=0, T=0, perm=Z, off=Z, E=1, x=Z, y=Z)


def test_binding_refuses_host_tensors(M):
    import torch

    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(M.MoeError) as ei:
        M.moe_norm_forward(x, M.MOE_BF16, M.MOE_NORM_RMS, torch.ones(64), None, 1e-5, 4, 64, x.clone(), stream=0)
    assert ei.value.status == M.MOE_ERR_INVALID_ARG and "GPU" in ei.value.message
