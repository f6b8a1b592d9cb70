"""The root-mean-square norm and its backward pass on the GPU against the formulas in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import ffn_ref as R  # noqa: E402

DEV = "cuda:0"
BF, F = torch.bfloat16, torch.float32

# A row's h^2 are added in fp32, at most 64 of a lane one after another, 6 steps across the
# wave and 16 waves: the sum is off by 2^-24 * 90 of itself at most, rstd by half of that and 3
# roundings, y by 2 more: 50 * 2^-24.
REL = 50 * 2.0 ** -24


def make(T, K, dtype, seed=0, wide=0, residual=True, weight=F):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def n(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    x = n(T, K + wide).to(dtype)[:, :K]
    r = (2 * n(T, K + wide)).to(dtype)[:, :K] if residual else None
    w = (1 + 0.3 * n(K)).to(weight) if weight is not None else None
    return x, r, w, n


def check(x, r, w, out, fmt, eps=1e-6):
    q, s, h, y, rstd = out
    want_h, want_r, want_y = R.norm(x, w, r, eps)
    assert torch.equal(h, want_h)
    if rstd is not None:
        assert ((rstd.double() - want_r).abs() <= REL * want_r).all()
    if q is not None:
        R.check_codes(q, s, want_y, REL * want_y.abs(), fmt)
        R.check_codes_sharp(q, s, want_y, 2 * REL, fmt)
    if y is not None:
        assert ((y.double() - want_y).abs() <= (2.0 ** -8 + 2 * REL) * want_y.abs()).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,K", [(1, 128), (1, 7168), (3, 512), (5, 640), (2, 2048), (7, 2176), (64, 4096),
                                 (9, 4224), (300, 7168), (3, 8320), (2, 16384), (2, 16512), (2, 32768),
                                 (2, 32896), (1, 65536), (2000, 128), (1027, 1536)])
def test_norm(T, K, dtype, fmt):
    x, r, w, _ = make(T, K, dtype, seed=K)
    check(x, r, w, dg.dg_rms_norm_fp8(x, w, residual=r, fmt=fmt, bf16=True, save=True), fmt)
    check(x, None, None, dg.dg_rms_norm_fp8(x, fmt=fmt), fmt)


@pytest.mark.parametrize("weight", [None, BF, F])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("wide", [0, 8, 24])
def test_norm_strides_and_options(weight, residual, wide):
    x, r, w, _ = make(37, 1152, BF, residual=residual, weight=weight, wide=wide)
    check(x, r, w, dg.dg_rms_norm_fp8(x, w, residual=r, save=True), "e4m3")
    out = dg.dg_rms_norm_fp8(x, w, residual=r, codes=False, bf16=True)
    assert out[0] is None and out[1] is None and out[4] is None
    check(x, r, w, out, "e4m3")
    y = torch.full((37, 1160), 7.0, device=DEV, dtype=BF)
    check(x, r, w, dg.dg_rms_norm_fp8(x, w, residual=r, Y=y[:, :1152]), "e4m3")
    assert (y[:, 1152:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F])
def test_norm_in_place(dtype):
    """H may be X or the residual, inside wider rows whose rest stays."""
    x, r, w, _ = make(65, 768, dtype, wide=16)
    want = dg.dg_rms_norm_fp8(x, w, residual=r, save=True)
    for k in range(2):
        base = (x if k == 0 else r)
        whole = torch.full((65, 784), -3.0, device=DEV, dtype=dtype)
        mine = whole[:, :768]
        mine.copy_(base)
        args = dict(X=mine, residual=r) if k == 0 else dict(X=x, residual=mine)
        got = dg.dg_rms_norm_fp8(weight=w, H=mine, save=True, **args)
        assert got[2] is mine and (whole[:, 768:] == -3).all()
        for a, b in zip(got, want):
            assert a is b is None or torch.equal(a.float(), b.float())


def test_norm_eps_zero_rows_and_sizes():
    x = torch.zeros(4, 256, device=DEV)
    x[1, 3] = 1e-3
    x[2] = 1e-4 * torch.arange(256, device=DEV)
    x[3, :128] = 5.0
    for eps in (1e-5, 1e-2):
        out = dg.dg_rms_norm_fp8(x, eps=eps, bf16=True, save=True)
        check(x, None, None, out, "e4m3", eps)
        assert (out[1][0] == 1).all() and (out[0][0].float() == 0).all()       # a block of zeros: scale 1
        assert out[1][3, 1] == 1
    for T in (0, 1):
        q, s, h, y, rstd = dg.dg_rms_norm_fp8(torch.zeros(T, 128, device=DEV), bf16=True, save=True)
        assert q.shape == (T, 128) and s.shape == (T, 1) and y.shape == (T, 128) and rstd.shape == (T,)


def test_norm_nan_and_infinity_stay_in_their_rows():
    x, r, w, _ = make(8, 512, BF)
    want = dg.dg_rms_norm_fp8(x, w, residual=r, bf16=True, save=True)
    x[2, 100] = float("nan")
    r[5, 300] = float("inf")
    q, s, h, y, rstd = dg.dg_rms_norm_fp8(x, w, residual=r, bf16=True, save=True)
    others = [0, 1, 3, 4, 6, 7]
    for a, b in zip((q, s, h, y, rstd), want):
        assert torch.equal(a[others].float(), b[others].float())
    assert s[2].isnan().all() and y[2].isnan().all()
    # finite values over an infinite root mean square are zero, the infinity itself is NaN
    assert rstd[5] == 0 and y[5, 300].isnan() and (y[5, :300] == 0).all()
    assert s[5, 2].isnan() and (s[5, [0, 1, 3]] == 1).all()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,K", [(1, 128), (1, 7168), (3, 640), (5, 2048), (7, 2176), (517, 4096), (9, 4224),
                                 (2100, 7168), (3, 8320), (4, 16384), (2, 32768), (2, 32896), (1, 65536),
                                 (3000, 128)])
def test_backward(T, K, dtype):
    for residual, weight in ((True, F), (False, BF), (True, None)):
        x, dh, w, n = make(T, K, dtype, seed=T, residual=residual, weight=weight, wide=8)
        dy = (0.1 * n(T, K)).to(dtype)
        _, rstd, _ = R.norm(x, w)
        rstd = rstd.float()
        gx, gw = dg.dg_rms_norm_backward(dy, x, rstd, w, grad_h=dh)
        want, want_w, mag, mag_w = R.norm_backward(dy, x, rstd, w, dh)
        # sums over K as for the norm (90 steps), a few roundings around them, one to the type
        assert ((gx.double() - want).abs() <= HALF(dtype) * want.abs() + 100 * 2.0 ** -24 * mag).all()
        if weight is None:
            assert gw is None
        else:
            # a sum over rows: T roundings at most, and 3 of each product
            assert ((gw.double() - want_w).abs() <= (T + 4) * 2.0 ** -24 * mag_w).all()
        assert dg.dg_rms_norm_backward(dy, x, rstd, w, grad_h=dh, grad_weight=False)[1] is None


def HALF(dtype):
    return R.HALF[dtype] * (1 + 2.0 ** -7)


def test_backward_in_place_and_empty():
    x, dh, w, n = make(130, 1024, BF)
    dy = n(130, 1024).to(BF)
    rstd = dg.dg_rms_norm_fp8(x, w, codes=False, save=True)[4]
    want = dg.dg_rms_norm_backward(dy, x, rstd, w, grad_h=dh)
    for which in range(2):
        a, b = dy.clone(), dh.clone()
        got = dg.dg_rms_norm_backward(a, x, rstd, w, grad_h=b, grad_x=(a, b)[which])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    gw = torch.full((1024,), 3.0, device=DEV)
    e = torch.empty(0, 1024, device=DEV, dtype=BF)
    got = dg.dg_rms_norm_backward(e, e, torch.empty(0, device=DEV), w, grad_weight=gw)
    assert got[0].shape == (0, 1024) and (gw == 0).all()


def test_backward_against_differences():
    """The GPU's gradient against differences of the norm in 64 bits, along directions."""
    x, _, w, n = make(6, 384, F, residual=False)
    dy = n(6, 384)
    rstd = dg.dg_rms_norm_fp8(x, w, codes=False, save=True)[4]
    gx, gw = dg.dg_rms_norm_backward(dy, x, rstd, w)
    for _ in range(3):
        d, dw, h = n(6, 384).double(), n(384).double(), 1e-5
        x64, w64 = x.double(), w.double()

        def f(a, b):
            return float((R.norm(a, b)[2] * dy.double()).sum())

        want = (f(x64 + h * d, w64 + h * dw) - f(x64 - h * d, w64 - h * dw)) / (2 * h)
        got = float((gx.double() * d).sum() + (gw.double() * dw).sum())
        size = float((gx.double() * d).abs().sum() + (gw.double() * dw).abs().sum())
        assert abs(got - want) <= 1e-5 * size


def test_same_bits_again_and_on_another_stream():
    x, r, w, n = make(1500, 7168, BF)
    dy = n(1500, 7168).to(BF)
    out = dg.dg_rms_norm_fp8(x, w, residual=r, save=True)
    back = dg.dg_rms_norm_backward(dy, out[2], out[4], w, grad_h=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2 = dg.dg_rms_norm_fp8(x, w, residual=r, save=True, stream=side)
    back2 = dg.dg_rms_norm_backward(dy, out2[2], out2[4], w, grad_h=r, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(out + back, out2 + back2):
        assert a is b is None or torch.equal(a.float(), b.float())


def test_graph():
    """Both passes captured together and replayed on new values, other work between."""
    x, r, w, n = make(700, 2048, BF)
    dy = n(700, 2048).to(BF)

    def step():
        q, s, h, _, rstd = dg.dg_rms_norm_fp8(x, w, residual=r, save=True)
        return (q, s, h, rstd) + dg.dg_rms_norm_backward(dy, h, rstd, w, grad_h=r)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(n(700, 2048))
        dy.copy_(n(700, 2048))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a.float(), b.float())


def test_refusals():
    x = torch.zeros(4, 256, device=DEV)
    w = torch.zeros(256, device=DEV)
    with pytest.raises(ValueError, match="must be on a GPU"):
        dg.dg_rms_norm_fp8(x.cpu())
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        dg.dg_rms_norm_fp8(x.half())
    with pytest.raises(ValueError, match="2-D"):
        dg.dg_rms_norm_fp8(x[0])
    with pytest.raises(ValueError, match="dense rows"):
        dg.dg_rms_norm_fp8(x.t().contiguous().t())
    with pytest.raises(dg.DGError, match="SHAPE"):
        dg.dg_rms_norm_fp8(x[:, :200])
    with pytest.raises(dg.DGError, match="SHAPE"):
        dg.dg_rms_norm_fp8(torch.zeros(4, 260, device=DEV)[:, :256])           # stride not 8 n
    with pytest.raises(dg.DGError, match="ALIGN"):
        dg.dg_rms_norm_fp8(torch.zeros(4, 264, device=DEV)[:, 2:258])
    with pytest.raises(dg.DGError, match="SHAPE"):
        dg.dg_rms_norm_fp8(torch.zeros(1, 65664, device=DEV))
    with pytest.raises(ValueError, match="weight must have shape"):
        dg.dg_rms_norm_fp8(x, w[:128])
    with pytest.raises(TypeError, match="residual must be"):
        dg.dg_rms_norm_fp8(x, residual=x.bfloat16())
    with pytest.raises(ValueError, match="with a residual"):
        dg.dg_rms_norm_fp8(x, H=x)
    with pytest.raises(ValueError, match="codes=True"):
        dg.dg_rms_norm_fp8(x, codes=False, S=w)
    with pytest.raises(ValueError, match="unknown fp8 format"):
        dg.dg_rms_norm_fp8(x, fmt="e3m4")
    with pytest.raises(ValueError, match="contradicts"):
        dg.dg_rms_norm_fp8(x, Q=torch.zeros(4, 256, device=DEV, dtype=torch.uint8).view(torch.float8_e5m2))
    rstd = torch.ones(4, device=DEV)
    with pytest.raises(TypeError, match="H must be"):
        dg.dg_rms_norm_backward(x, x.bfloat16(), rstd)
    with pytest.raises(ValueError, match="rstd must have shape"):
        dg.dg_rms_norm_backward(x, x, rstd[:3])
    with pytest.raises(dg.DGError, match="WORKSPACE"):
        dg.dg_rms_norm_backward(x, x, rstd, w, workspace=torch.empty(16, device=DEV))
