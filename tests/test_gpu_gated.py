"""The gated feed-forward block's first half and its backward pass on the GPU against the
formulas in 64 bits: the dense, contiguous and masked forms, and the 8-bit checkpoint."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import ffn_ref as R  # noqa: E402

DEV = "cuda:0"
BF, F = torch.bfloat16, torch.float32

# A projection's sum of K products: those of a 128-block are exact in fp32 and summed with at
# most 128 roundings of 2^-24 of the running sum, which their magnitudes' sum bounds; then a
# product with the scales and an addition for each of the K / 128 blocks.
SUM = 2.0 ** -24
# The sigmoid: exp and the reciprocal to an ulp each, its argument rounded (2^-23 |z|, |z| up
# to about 20 where it matters), three products.
ACT = 2.0 ** -18


def gen(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return g, lambda *s: torch.randn(*s, generator=g, device=DEV)


def weights(n, K, N, G=None, fmt="e4m3"):
    return R.quantise_weight(n(*(() if G is None else (G,)), 2 * N, K) * K ** -0.5, fmt)


def check(H, sH, GU, sGU, x, w, act, fmt, what):
    """Rows x of one group (values in 64 bits) against its weight's values."""
    N = w.shape[0] // 2
    gu = x @ w.t()
    err = SUM * (128 + 3 + w.shape[1] // 128) * (x.abs() @ w.abs().t())
    g, u, eg, eu = gu[:, :N], gu[:, N:], err[:, :N], err[:, N:]
    h = R.gated(g, u, act)
    # |act'| is below 1.13; products of errors are covered by the second eg
    eh = 1.13 * eg * (u.abs() + eu) + (g.abs() + eg) * eu + ACT * h.abs()
    R.check_codes(H, sH, h, eh, fmt, what + " h")
    if GU is not None:
        R.check_codes(GU, sGU, gu, err, fmt, what + " gate and up")


FORMATS = [("e4m3", "e4m3", "e4m3"), ("e5m2", "e4m3", "e4m3"), ("e4m3", "e5m2", "e5m2"), ("e5m2", "e5m2", "e4m3")]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (1, 2048, 7168), (2, 128, 2048), (7, 384, 256), (16, 256, 1024),
                                   (17, 1024, 640), (31, 128, 384), (33, 640, 128), (64, 2048, 512),
                                   (65, 256, 896), (128, 1152, 256), (129, 256, 384), (255, 128, 128),
                                   (300, 512, 1024), (517, 896, 640), (1500, 4096, 256), (2049, 4352, 384)])
def test_dense(M, N, K, act):
    g, n = gen(M + N + K)
    for save in (False, True):
        fa, fb, fmt = FORMATS[(M + N // 128 + save) % 4]
        a, sa = R.quantise(n(M, K), fa)
        b, sb = weights(n, K, N, fmt=fb)
        out = dg.dg_gated_fp8_nt(a, sa, b, sb, activation=act, fmt=fmt, save=save)
        assert (out[2] is None) == (out[3] is None) == (not save)
        check(*out, R.values(a, sa), R.weight_values(b, sb), act, fmt, f"{M}x{N}x{K} {fa} {fb} {fmt}")


@pytest.mark.parametrize("fa,fb,fmt", FORMATS)
@pytest.mark.parametrize("M", [3, 70, 200, 3000])
def test_formats(M, fa, fb, fmt):
    g, n = gen(M)
    a, sa = R.quantise(n(M, 512), fa)
    b, sb = weights(n, 512, 2816, fmt=fb)
    by_dtype = dg.dg_gated_fp8_nt(a, sa, b, sb, fmt=fmt, save=True)
    by_name = dg.dg_gated_fp8_nt(a.view(torch.uint8), sa, b.view(torch.uint8), sb, a_format=fa, b_format=fb,
                                 fmt=fmt, save=True)
    check(*by_dtype, R.values(a, sa), R.weight_values(b, sb), "silu", fmt, "formats")
    for p, q in zip(by_dtype, by_name):
        assert torch.equal(p.float(), q.float())


@pytest.mark.parametrize("M", [1, 5, 40, 100, 200, 2100])
def test_whole_numbers(M):
    """Small whole numbers and scales of powers of two: both projections are exact in fp32, so
    every code is the one of the value, but for the activation's own error near a border."""
    g, n = gen(9)
    K, N = 384, 3200
    a = torch.randint(-3, 4, (M, K), generator=g, device=DEV).float()
    b = torch.randint(-2, 3, (2 * N, K), generator=g, device=DEV).float()
    sa = torch.exp2(torch.randint(-6, -3, (M, K // 128), generator=g, device=DEV).float())
    sb = torch.exp2(torch.randint(-3, 0, (2 * N // 128, K // 128), generator=g, device=DEV).float())
    a, b = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
    H, sH, GU, sGU = dg.dg_gated_fp8_nt(a, sa, b, sb, save=True)
    gu = R.values(a, sa) @ R.weight_values(b, sb).t()
    R.check_codes_sharp(GU, sGU, gu, 2.0 ** -23, "e4m3", "gate and up")
    R.check_codes_sharp(H, sH, R.gated(gu[:, :N], gu[:, N:], "silu"), ACT, "e4m3", "h")
    amax = gu.abs().view(M, -1, 128).amax(-1)
    # the scale: one division, rounded (torch's own by a number is a product with its inverse)
    assert torch.equal(sGU, torch.where(amax == 0, 1.0, amax / 448).float())


def test_zero_rows_and_a_shared_scale():
    """A row of zeros has zero codes and scale 1; an element of the other half of a 128-block
    decides its scale."""
    g, n = gen(4)
    a, sa = R.quantise(n(140, 256))
    a.view(torch.uint8)[3] = 0
    b, sb = R.quantise_weight(n(512, 256) * 0.1)
    w = b.float()
    w[100] *= 8
    b = w.clamp(-448, 448).to(b.dtype)
    H, sH, GU, sGU = dg.dg_gated_fp8_nt(a, sa, b, sb, save=True)
    for c, s in ((H, sH), (GU, sGU)):
        assert (c[3].float() == 0).all() and (s[3] == 1).all()
    check(H, sH, GU, sGU, R.values(a, sa), R.weight_values(b, sb), "silu", "e4m3", "zero row")


def _segments(sizes, tail=0):
    """group_idx of segments (group, rows) padded to 128 rows with -1, and `tail` more rows."""
    idx = []
    for grp, rows in sizes:
        idx += [grp] * rows + [-1] * (-rows % 128)
    return torch.tensor(idx + [-1] * tail, dtype=torch.int32, device=DEV)


SEGMENTS = [[(0, 100)], [(2, 1), (0, 128), (1, 200)], [(1, 130), (3, 5), (0, 256), (1, 77)],
            [(g, 100 + 60 * g) for g in range(5)], [(3, 2000), (0, 1500), (2, 999)], [(0, 3000), (1, 10)]]


@pytest.mark.parametrize("N,K", [(256, 384), (2944, 128)], ids=["narrow", "wide"])
@pytest.mark.parametrize("case", range(len(SEGMENTS)))
def test_contiguous(case, N, K):
    G = 5
    idx = _segments(SEGMENTS[case], tail=(0, 61)[case % 2])
    if case == 2:
        idx[10:20] = 4                                # rows of another group than their block's
        idx[300] = G                                  # out of range
    M = idx.numel()
    g, n = gen(case)
    a, sa = R.quantise(n(M, K))
    b, sb = weights(n, K, N, G)
    live = R.written(idx, G)
    a.view(torch.uint8)[~live] = 0x7F                # rows that are not written may hold anything
    sa[~live] = float("nan")
    H = torch.full((M, N), 0x55, dtype=torch.uint8, device=DEV)
    sH = torch.full((M, N // 128), -7.0, device=DEV)
    GU = torch.full((M, 2 * N), 0x55, dtype=torch.uint8, device=DEV)
    sGU = torch.full((M, N // 64), -7.0, device=DEV)
    out = dg.dg_grouped_gated_fp8_contiguous(a, sa, b, sb, idx, H, sH, GU=GU, sGU=sGU)
    assert (H[~live] == 0x55).all() and (GU[~live] == 0x55).all()
    assert (sH[~live] == -7).all() and (sGU[~live] == -7).all()
    for i in range(G):
        at = live & (idx == i)
        if at.any():
            check(*(o[at] for o in out), R.values(a[at], sa[at]), R.weight_values(b[i], sb[i]), "silu", "e4m3",
                  f"group {i}")
    plain = dg.dg_grouped_gated_fp8_contiguous(a, sa, b, sb, idx)
    assert torch.equal(plain[0][live].float(), out[0][live].float()) and torch.equal(plain[1][live], sH[live])
    assert (plain[0][~live].float() == 0).all() and plain[2] is None


@pytest.mark.parametrize("G,cap,counts", [(1, 1, [1]), (3, 16, [16, 0, 5]), (4, 64, [0, 64, 33, 1]),
                                          (2, 100, [99, 100]), (5, 128, [128, 0, 127, 3, 64]),
                                          (3, 200, [200, 129, 128]), (2, 513, [513, 257]), (4, 300, [0, 0, 0, 0]),
                                          (3, 40, [-5, 99, 40]), (70, 20, list(range(-20, 50)))])
@pytest.mark.parametrize("N,K", [(128, 256), (1408, 384)])
def test_masked(G, cap, counts, N, K):
    g, n = gen(G + cap)
    a, sa = R.quantise(n(G, cap, K))
    b, sb = weights(n, K, N, G)
    rows = [max(0, min(c, cap)) for c in counts]
    live = torch.arange(cap, device=DEV) < torch.tensor(rows, device=DEV)[:, None]
    a.view(torch.uint8)[~live] = 0x7F
    sa[~live] = float("nan")
    H = torch.full((G, cap, N), 0x55, dtype=torch.uint8, device=DEV)
    sH = torch.full((G, cap, N // 128), -7.0, device=DEV)
    mm = torch.tensor(counts, dtype=torch.int32, device=DEV)
    out = dg.dg_grouped_gated_fp8_masked(a, sa, b, sb, mm, H, sH, activation="gelu")
    assert out[2] is None and out[3] is None
    assert (H[~live] == 0x55).all() and (sH[~live] == -7).all()
    for i, r in enumerate(rows):
        if r:
            check(out[0][i, :r], out[1][i, :r], None, None, R.values(a[i, :r], sa[i, :r]),
                  R.weight_values(b[i], sb[i]), "gelu", "e4m3", f"group {i}")


def test_empty():
    b, sb = torch.zeros(512, 256, device=DEV, dtype=torch.uint8), torch.ones(4, 2, device=DEV)
    a, sa = torch.zeros(0, 256, device=DEV, dtype=torch.uint8), torch.zeros(0, 2, device=DEV)
    H, sH, GU, sGU = dg.dg_gated_fp8_nt(a, sa, b, sb, save=True)
    assert H.shape == (0, 256) and GU.shape == (0, 512) and sGU.shape == (0, 4)


@pytest.mark.parametrize("M", [1, 60, 129, 5000])
def test_same_bits_again_graph_and_stream(M):
    g, n = gen(M)
    a, sa = R.quantise(n(M, 512))
    b, sb = weights(n, 512, 1280)
    want = dg.dg_gated_fp8_nt(a, sa, b, sb, save=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dg.dg_gated_fp8_nt(a, sa, b, sb, save=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = dg.dg_gated_fp8_nt(a, sa, b, sb, save=True)
    for p, q in zip(got, want):
        assert torch.equal(p.float(), q.float())
    for _ in range(3):
        a2, sa2 = R.quantise(n(M, 512))
        a.view(torch.uint8).copy_(a2.view(torch.uint8))
        sa.copy_(sa2)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(held, dg.dg_gated_fp8_nt(a, sa, b, sb, save=True)):
            assert torch.equal(p.float(), q.float())


def test_rows_beyond_two_to_the_31_bytes():
    """The last rows of outputs and checkpoints whose offsets pass 32 bits."""
    M, N, K = 70000, 16384, 128
    g, n = gen(8)
    a, sa = R.quantise(n(M, K))
    b, sb = weights(n, K, N)
    H, sH, GU, sGU = dg.dg_gated_fp8_nt(a, sa, b, sb, save=True)
    w = R.weight_values(b, sb)
    for at in (slice(0, 40), slice(M // 2, M // 2 + 40), slice(M - 40, M)):
        check(H[at], sH[at], GU[at], sGU[at], R.values(a[at], sa[at]), w, "silu", "e4m3", str(at))
    dh = n(40, N).to(BF)
    whole = torch.zeros(M, N, device=DEV, dtype=BF)
    whole[M - 40:] = dh
    D, sD = dg.dg_gated_backward(whole, GU, sGU)
    part = dg.dg_gated_backward(dh, GU[M - 40:].clone(), sGU[M - 40:].clone())
    assert torch.equal(D[M - 40:].float(), part[0].float()) and torch.equal(sD[M - 40:], part[1])


# ------------------------------------------------------------------------ backward pass
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gu_fmt,fmt", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2")])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,N", [(1, 128), (3, 256), (17, 640), (130, 2048), (517, 1152)])
def test_backward(T, N, dtype, gu_fmt, fmt, act):
    g, n = gen(T + N)
    gu, sgu = R.quantise(2 * n(T, 2 * N), gu_fmt)
    dh = (0.01 * n(T, N)).to(dtype)
    D, sD = dg.dg_gated_backward(dh, gu, sgu, activation=act, fmt=fmt)
    v = R.values(gu, sgu)
    x, u = v[:, :N], v[:, N:]
    want = R.gated_backward(dh.double(), x, u, act)
    # as the forward pass; the derivative's two parts may cancel, so its error goes by their sum
    s, dz = R.sigmoid_of(x, act)
    mag = torch.cat([(dh.double() * u).abs() * (s + (x * s * (1 - s) * dz).abs()), (dh.double() * x * s).abs()], 1)
    # near 1, 1 - s is off by the error of s itself: |g dz| (2^-22) beside it
    mag[:, :N] += (dh.double() * u * x * s * dz).abs() * 2.0 ** -4
    R.check_codes(D, sD, want, ACT * mag, fmt, "D")


def test_backward_far_from_zero():
    """Gates whose exponentials leave fp32's range: the derivative is zero or one."""
    x = torch.tensor([-3e4, -200.0, -90.0, 90.0, 200.0, 3e4, 0.0, -0.0], device=DEV).repeat(16)
    gu = torch.cat([x, torch.ones(128, device=DEV)])[None]
    for act in ("silu", "gelu"):
        for scale in (1.0, 2.0 ** 60):
            q, s = R.quantise(gu, "e5m2")
            s[:, 0] *= scale
            D, sD = dg.dg_gated_backward(torch.ones(1, 128, device=DEV), q, s, activation=act)
            v = R.values(D, sD)[0]
            assert torch.isfinite(v).all()
            far = x.abs() >= 90
            # 448 times the scale 1 / 448, which is rounded to fp32
            assert ((v[:128] - (x > 0).double()).abs()[far] <= 2.0 ** -24).all()


@pytest.mark.parametrize("case", range(len(SEGMENTS)))
def test_backward_contiguous(case):
    G, N = 5, 384
    idx = _segments(SEGMENTS[case], tail=61)
    idx[5:9] = -1
    M = idx.numel()
    g, n = gen(case)
    live = R.written(idx, G)
    gu, sgu = R.quantise(n(M, 2 * N))
    dh = n(M, N).to(BF)
    gu.view(torch.uint8)[~live] = 0x7F
    sgu[~live] = float("nan")
    dh[~live] = float("nan")
    D = torch.full((M, 2 * N), 0x55, dtype=torch.uint8, device=DEV)
    sD = torch.full((M, N // 64), -7.0, device=DEV)
    out = dg.dg_gated_backward(dh, gu, sgu, D, sD, group_idx=idx, groups=G)
    assert (D[~live] == 0x55).all() and (sD[~live] == -7).all()
    alone = dg.dg_gated_backward(dh[live], gu.view(torch.uint8)[live].view(gu.dtype), sgu[live])
    assert torch.equal(out[0].view(torch.uint8)[live], alone[0].view(torch.uint8)) and torch.equal(sD[live], alone[1])


def test_backward_in_place():
    g, n = gen(2)
    gu, sgu = R.quantise(n(150, 1024))
    dh = n(150, 512).to(BF)
    want = dg.dg_gated_backward(dh, gu, sgu)
    got = dg.dg_gated_backward(dh, gu, sgu, gu, sgu)
    assert got[0] is gu and got[1] is sgu
    assert torch.equal(got[0].float(), want[0].float()) and torch.equal(got[1], want[1])


def test_backward_against_differences():
    """Along directions of g and u: the codes' values against differences of h in 64 bits, off by
    what their rounding allows."""
    g, n = gen(6)
    N = 256
    gu, sgu = R.quantise(n(20, 2 * N))
    dh = n(20, N)
    v = R.values(gu, sgu)
    D, sD = dg.dg_gated_backward(dh, gu, sgu)
    got = R.values(D, sD)
    for _ in range(3):
        d, h = n(20, 2 * N).double(), 1e-5

        def f(a):
            return float((R.gated(a[:, :N], a[:, N:], "silu") * dh.double()).sum())

        want = (f(v + h * d) - f(v - h * d)) / (2 * h)
        allowed = (d.abs() * (got.abs() * 2.0 ** -4 + 2.0 ** -10 * sD.double().repeat_interleave(128, 1))).sum()
        assert abs(float((got * d).sum()) - want) <= 1.1 * float(allowed)


def test_refusals():
    a, sa = torch.zeros(4, 256, device=DEV, dtype=torch.uint8), torch.ones(4, 2, device=DEV)
    b, sb = torch.zeros(512, 256, device=DEV, dtype=torch.uint8), torch.ones(4, 2, device=DEV)
    f = dg.dg_gated_fp8_nt
    with pytest.raises(ValueError, match="must be on a GPU"):
        f(a.cpu(), sa, b, sb)
    with pytest.raises(TypeError, match="uint8"):
        f(a.float(), sa, b, sb)
    with pytest.raises(ValueError, match="multiple of 128"):
        f(a, sa, b[:384], sb[:3])
    with pytest.raises(ValueError, match="sB must have shape"):
        f(a, sa, b, sb[:2])
    with pytest.raises(ValueError, match="B must have shape"):
        f(a, sa, torch.zeros(512, 384, device=DEV, dtype=torch.uint8), sb)
    with pytest.raises(ValueError, match="unknown activation"):
        f(a, sa, b, sb, activation="relu")
    with pytest.raises(ValueError, match="unknown fp8 format"):
        f(a, sa, b, sb, fmt="fp8")
    with pytest.raises(dg.DGError, match="SHAPE"):
        f(torch.zeros(4, 200, device=DEV, dtype=torch.uint8), torch.ones(4, 2, device=DEV),
          torch.zeros(512, 200, device=DEV, dtype=torch.uint8), sb)
    with pytest.raises(ValueError, match="H must have shape"):
        f(a, sa, b, sb, torch.zeros(4, 512, device=DEV, dtype=torch.uint8))
    with pytest.raises(ValueError, match="group_idx must have shape"):
        dg.dg_grouped_gated_fp8_contiguous(a, sa, b[None], sb[None], torch.zeros(3, device=DEV, dtype=torch.int32))
    with pytest.raises(ValueError, match="groups"):
        dg.dg_grouped_gated_fp8_masked(a[None], sa[None], b.view(1, 512, 256).expand(2, 512, 256),
                                       sb[None], torch.zeros(1, device=DEV, dtype=torch.int32))
    with pytest.raises(ValueError, match="contiguous"):
        f(torch.zeros(256, 4, device=DEV, dtype=torch.uint8).t(), sa, b, sb)
    gb = dg.dg_gated_backward
    gu, sgu = torch.zeros(4, 512, device=DEV, dtype=torch.uint8), torch.ones(4, 4, device=DEV)
    with pytest.raises(TypeError, match="grad_H must be"):
        gb(torch.zeros(4, 256, device=DEV, dtype=torch.float16), gu, sgu)
    with pytest.raises(ValueError, match="GU must have shape"):
        gb(torch.zeros(4, 128, device=DEV), gu, sgu)
    with pytest.raises(dg.DGError, match="SHAPE"):
        gb(torch.zeros(4, 256, device=DEV), gu, sgu, groups=0)
