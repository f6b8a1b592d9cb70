"""Host-side checks of the feed-forward operators in 8 bits that need no GPU: every documented
error code comes before any device state is touched, in the documented order."""
import os

import pytest

A16, A8, A4, A2 = 0x10000, 0x20008, 0x30004, 0x40002      # fake addresses: never dereferenced
SHAPE, FORMAT, NULL, ALIGN, WORKSPACE, DEVICE = 2, 7, 1, 3, 4, 5


@pytest.fixture(scope="module")
def native():
    from moe_grouped_gemm_lhs_amd import binding, build, moe_ops
    if not (os.path.exists(binding.LIB_PATH) and os.path.exists(build.MARSHAL)):
        if not os.path.exists(build.HIPCC):
            pytest.skip("not built and hipcc unavailable")
        build.build()
    return moe_ops._load_native()


def norm(n, X=A16, dtype=0, ldx=256, r=None, ldr=0, w=None, wd=0, H=None, ldh=0, Q=A8, S=A4, fmt=0, Y=None, ldy=0,
         rstd=None, T=4, K=256):
    return n.dg_rms_norm_fp8(X, dtype, ldx, r, ldr, w, wd, 1e-6, H, ldh, Q, S, fmt, Y, ldy, rstd, T, K, None)


def test_norm_codes(native):
    for bad in (dict(K=200), dict(K=0), dict(K=-128), dict(K=65536 + 128, ldx=1 << 20), dict(T=-1), dict(T=1 << 31),
                dict(ldx=248), dict(ldx=260), dict(r=A16, H=A16, ldr=255, ldh=256), dict(r=A16, H=A16, ldr=256),
                dict(Y=A16, ldy=128)):
        assert norm(native, **bad) == SHAPE, bad
    assert norm(native, dtype=2) == FORMAT
    assert norm(native, w=A16, wd=5) == FORMAT
    assert norm(native, fmt=2) == FORMAT
    assert norm(native, fmt=2, K=200) == SHAPE            # shapes first
    assert norm(native, T=0, X=None, Q=None) == 0
    for bad in (dict(X=None), dict(Q=None), dict(S=None), dict(r=A16, ldr=256, ldh=256), dict(H=A16)):
        assert norm(native, **bad) == NULL, bad
    for bad in (dict(X=A8), dict(Q=A4), dict(S=A2), dict(w=A8), dict(rstd=A2), dict(Y=A8, ldy=256),
                dict(r=A8, H=A16, ldr=256, ldh=256), dict(r=A16, H=A8, ldr=256, ldh=256)):
        assert norm(native, **bad) == ALIGN, bad


def norm_back(n, dy=A16, dtype=0, ld=256, H=A16, ldh=256, rstd=A4, w=None, wd=0, dh=None, ldd=0, dx=A16, ldx=256,
              dw=None, T=4, K=256, ws=None, wsb=0):
    return n.dg_rms_norm_backward(dy, dtype, ld, H, ldh, rstd, w, wd, dh, ldd, dx, ldx, dw, T, K, ws, wsb, None)


def test_norm_backward_codes(native):
    for bad in (dict(K=100), dict(T=-1), dict(ld=128), dict(ldh=252), dict(ldx=255), dict(dh=A16, ldd=0)):
        assert norm_back(native, **bad) == SHAPE, bad
    assert norm_back(native, dtype=3) == FORMAT
    assert norm_back(native, w=A16, wd=-1) == FORMAT
    assert norm_back(native, T=0, dy=None, H=None, rstd=None, dx=None) == 0
    for bad in (dict(dy=None), dict(H=None), dict(rstd=None), dict(dx=None)):
        assert norm_back(native, **bad) == NULL, bad
    for bad in (dict(dy=A8), dict(H=A8), dict(rstd=A2), dict(dx=A8), dict(w=A8), dict(dw=A2), dict(dh=A8, ldd=256)):
        assert norm_back(native, **bad) == ALIGN, bad
    need = native.dg_rms_norm_backward_workspace_bytes(4, 256)
    assert need > 0 and native.dg_rms_norm_backward_workspace_bytes(4, 200) == 0
    for bad in (dict(), dict(ws=A16, wsb=need - 1), dict(ws=A8, wsb=need)):
        assert norm_back(native, dw=A4, **bad) == WORKSPACE, bad


def gated(n, kind="dense", A=A16, fa=0, sA=A4, B=A16, fb=0, sB=A4, rows_of=A4, H=A16, sH=A4, fmt=0, GU=None,
          sGU=None, act=0, rows=200, N=256, K=256, G=2, ws=A16, wsb=1 << 40):
    if kind == "dense":
        return n.dg_gated_fp8_nt(A, fa, sA, B, fb, sB, H, sH, fmt, GU, sGU, act, rows, N, K, ws, wsb, None)
    if kind == "masked":
        return n.dg_grouped_gated_fp8_masked(A, fa, sA, B, fb, sB, rows_of, H, sH, fmt, act, G, rows, N, K, ws, wsb,
                                             None)
    return n.dg_grouped_gated_fp8_contiguous(A, fa, sA, B, fb, sB, rows_of, H, sH, fmt, GU, sGU, act, rows, N, K, G,
                                             ws, wsb, None)


@pytest.mark.parametrize("kind", ["dense", "contiguous", "masked"])
def test_gated_codes(native, kind):
    for bad in (dict(K=0), dict(K=100), dict(K=1 << 23), dict(N=100), dict(N=-128), dict(N=(1 << 20) + 128),
                dict(rows=-1), dict(rows=1 << 31)):
        assert gated(native, kind, **bad) == SHAPE, bad
    if kind != "dense":
        assert gated(native, kind, G=0) == SHAPE
        assert gated(native, kind, rows_of=None) == NULL
        assert gated(native, kind, rows_of=A2) == ALIGN
    if kind == "masked":
        assert gated(native, kind, G=1 << 20, rows=1 << 14) == SHAPE
    for bad in (dict(fa=2), dict(fb=-1), dict(fmt=2), dict(act=2)):
        assert gated(native, kind, **bad) == FORMAT, bad
    assert gated(native, kind, rows=0, A=None) == 0 and gated(native, kind, N=0, B=None) == 0
    for bad in (dict(A=None), dict(sA=None), dict(B=None), dict(sB=None), dict(H=None), dict(sH=None)):
        assert gated(native, kind, **bad) == NULL, bad
    for bad in (dict(A=A8), dict(B=A8), dict(H=A8), dict(sA=A2), dict(sB=A2), dict(sH=A2)):
        assert gated(native, kind, **bad) == ALIGN, bad
    if kind != "masked":
        assert gated(native, kind, GU=A16) == NULL and gated(native, kind, sGU=A4) == NULL
        assert gated(native, kind, GU=A8, sGU=A4) == ALIGN and gated(native, kind, GU=A16, sGU=A2) == ALIGN


def back(n, dh=A16, dtype=0, GU=A16, gf=0, sGU=A4, idx=None, act=0, D=A16, sD=A4, fmt=0, T=4, N=256, G=1):
    return n.dg_gated_backward(dh, dtype, GU, gf, sGU, idx, act, D, sD, fmt, T, N, G, None)


def test_gated_backward_codes(native):
    for bad in (dict(T=-1), dict(N=100), dict(N=1 << 21), dict(G=0), dict(T=1 << 30, N=256 * 128)):
        assert back(native, **bad) == SHAPE, bad
    for bad in (dict(dtype=2), dict(gf=2), dict(fmt=-1), dict(act=7)):
        assert back(native, **bad) == FORMAT, bad
    assert back(native, T=0, dh=None) == 0 and back(native, N=0, D=None) == 0
    for bad in (dict(dh=None), dict(GU=None), dict(sGU=None), dict(D=None), dict(sD=None)):
        assert back(native, **bad) == NULL, bad
    for bad in (dict(dh=A8), dict(GU=A8), dict(sGU=A2), dict(D=A8), dict(sD=A2), dict(idx=A2)):
        assert back(native, **bad) == ALIGN, bad


def wgrad(n, grouped=False, P=A16, fp=0, sP=A4, Q=A16, fq=0, sQ=A4, idx=A4, dW=A16, dtype=0, acc=0, T=4, N=256, K=128,
          G=2, ws=A16, wsb=1 << 50):
    if grouped:
        return n.dg_grouped_wgrad_fp8_contiguous(P, fp, sP, Q, fq, sQ, idx, dW, dtype, acc, T, N, K, G, ws, wsb, None)
    return n.dg_wgrad_fp8(P, fp, sP, Q, fq, sQ, dW, dtype, acc, T, N, K, ws, wsb, None)


@pytest.mark.parametrize("grouped", [False, True])
def test_wgrad_codes(native, grouped):
    for bad in (dict(T=-1), dict(T=(1 << 31) - 1), dict(N=100), dict(K=-128), dict(K=(1 << 22) + 128),
                dict(N=1 << 22, K=1 << 22)):
        assert wgrad(native, grouped, **bad) == SHAPE, bad
    for bad in (dict(fp=2), dict(fq=3), dict(dtype=2)):
        assert wgrad(native, grouped, **bad) == FORMAT, bad
    assert wgrad(native, grouped, N=0, dW=None) == 0 and wgrad(native, grouped, T=0, acc=1, P=None) == 0
    for bad in (dict(P=None), dict(sP=None), dict(Q=None), dict(sQ=None), dict(dW=None), dict(T=0, dW=None)):
        assert wgrad(native, grouped, **bad) == NULL, bad
    for bad in (dict(P=A8), dict(Q=A8), dict(dW=A8), dict(sP=A2), dict(sQ=A2)):
        assert wgrad(native, grouped, **bad) == ALIGN, bad
    if grouped:
        assert wgrad(native, True, G=0) == SHAPE
        assert wgrad(native, True, idx=None) == NULL and wgrad(native, True, idx=A2) == ALIGN


def test_python_refuses_cpu_tensors(native):
    torch = pytest.importorskip("torch")
    import moe_grouped_gemm_lhs_amd as dg
    x, c, s = torch.zeros(4, 256), torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    for call in (lambda: dg.dg_rms_norm_fp8(x), lambda: dg.dg_rms_norm_backward(x, x, torch.zeros(4)),
                 lambda: dg.dg_gated_fp8_nt(c, s, c, s), lambda: dg.dg_gated_backward(x, c, s),
                 lambda: dg.dg_wgrad_fp8(c, s, c, s),
                 lambda: dg.dg_grouped_wgrad_fp8_contiguous(c, s, c, s, torch.zeros(4, dtype=torch.int32), 2)):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()


def test_gated_workspace_codes(native):
    """Few tiles need a workspace in every form, many none."""
    need = native.dg_gated_workspace_bytes(0, 64, 2048, 7168, 1)
    assert need > 0
    for bad in (dict(ws=None, wsb=0), dict(wsb=need - 1), dict(ws=A8)):
        assert gated(native, "dense", rows=64, N=2048, K=7168, **bad) == WORKSPACE, bad
    assert native.dg_gated_workspace_bytes(2, 256, 2048, 7168, 4) > 0
    assert native.dg_gated_workspace_bytes(0, 8192, 2048, 7168, 1) == 0
    assert native.dg_gated_workspace_bytes(1, 200, 2048, 7168, 4) > 0
    assert native.dg_gated_workspace_bytes(1, 8192, 2048, 7168, 4) == 0
    assert native.dg_gated_workspace_bytes(0, 64, 100, 7168, 1) == 0
    assert native.dg_gated_workspace_bytes(3, 64, 2048, 7168, 1) == 0
