"""Weights' gradients from 8-bit matrices on the GPU against the sums in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import ffn_ref as R  # noqa: E402

DEV = "cuda:0"
BF, F = torch.bfloat16, torch.float32


def make(T, N, K, p_fmt="e4m3", q_fmt="e4m3", seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=g, device=DEV)

    p, sp = R.quantise(0.01 * n(T, N) * torch.exp(n(T, 1)), p_fmt)
    q, sq = R.quantise(n(T, K), q_fmt)
    return p, sp, q, sq


def check(got, p, sp, q, sq, before=None, what=""):
    p, q = R.values(p, sp), R.values(q, sq)
    want, mag = p.t() @ q, p.abs().t() @ q.abs()
    if before is not None:
        want, mag = want + before.double(), mag + before.double().abs()
    # a product's factors are rounded to bf16 (2^-8, of both at most) and the sum of T products to
    # fp32 at each step; the result to its type
    tol = mag * (2.0 ** -7 + 2.0 ** -15 + (p.shape[0] + 4) * 2.0 ** -24) + R.HALF[got.dtype] * want.abs() * 1.01
    off = (got.double() - want).abs() - tol
    assert off.max() <= 0, f"{what}: off by {float(off.max()):.3g}"
    # such errors have either sign: together they are far smaller than each may be
    if want.numel() > 1000 and p.shape[0] > 16:
        rel = float((got.double() - want).norm() / want.norm())
        assert rel < 2.0 ** -7, f"{what}: {rel:.3g}"


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,N,K", [(1, 128, 128), (5, 256, 128), (63, 128, 384), (64, 384, 256), (65, 128, 128),
                                   (127, 256, 256), (128, 512, 128), (129, 128, 512), (300, 640, 384),
                                   (517, 1024, 256), (1093, 896, 640), (4096, 256, 128), (20000, 128, 128),
                                   (700, 4096, 1152)])
def test_dense(T, N, K, dtype):
    fp, fq = [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")][(T + N // 128) % 4]
    ops = make(T, N, K, fp, fq, seed=T)
    dw = dg.dg_wgrad_fp8(*ops, dtype=dtype)
    assert dw.dtype is dtype and dw.shape == (N, K)
    check(dw, *ops, what=f"{T} {N} {K} {fp} {fq}")
    old = torch.randn(N, K, device=DEV).to(dtype) * 0.01
    acc = old.clone()
    assert dg.dg_wgrad_fp8(*ops, acc, accumulate=True) is acc
    check(acc, *ops, before=old, what="accumulated")


@pytest.mark.parametrize("T,N,K", [(1, 128, 128), (77, 256, 384), (1000, 128, 256), (130, 1024, 1024),
                                   (5000, 256, 256)])
def test_whole_numbers(T, N, K):
    """Codes that are small whole numbers, scales that are powers of two: every product and sum
    is exact, and so is the result."""
    g = torch.Generator(device=DEV).manual_seed(T)
    p = torch.randint(-4, 5, (T, N), generator=g, device=DEV).float().to(torch.float8_e4m3fn)
    q = torch.randint(-4, 5, (T, K), generator=g, device=DEV).float().to(torch.float8_e5m2)
    sp = torch.exp2(torch.randint(-1, 2, (T, N // 128), generator=g, device=DEV).float())
    sq = torch.exp2(torch.randint(-1, 2, (T, K // 128), generator=g, device=DEV).float())
    want = R.values(p, sp).t() @ R.values(q, sq)
    assert torch.equal(dg.dg_wgrad_fp8(p, sp, q, sq).double(), want)
    idx = torch.where(torch.arange(T, device=DEV) // 128 % 2 == 0, 1, 0).int()
    got = dg.dg_grouped_wgrad_fp8_contiguous(p, sp, q, sq, idx, 3)
    for i in range(3):
        at = idx == i
        want = R.values(p[at], sp[at]).t() @ R.values(q[at], sq[at])
        assert torch.equal(got[i].double(), want)


def _segments(sizes, tail=0):
    idx = []
    for grp, rows in sizes:
        idx += [grp] * rows + [-1] * (-rows % 128)
    return torch.tensor(idx + [-1] * tail, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("sizes", [[(0, 100)], [(2, 1), (0, 128), (1, 200)], [(1, 130), (3, 5), (0, 256), (1, 77)],
                                   [(g, 100 + 60 * g) for g in range(5)], [(3, 2000), (0, 1500)],
                                   [(4, 64), (4, 65), (4, 128)], [(i % 5, 128) for i in range(150)]])
@pytest.mark.parametrize("tail", [0, 61])
def test_grouped(sizes, tail):
    G, N, K = 5, 256, 384
    idx = _segments(sizes, tail)
    idx[3:5] = -1
    if idx.numel() > 300:
        idx[290] = 4                                  # a row of another group than its block's
        idx[291] = G
    T = idx.numel()
    live = R.written(idx, G)
    p, sp, q, sq = make(T, N, K, seed=T)
    for c, s in ((p, sp), (q, sq)):                   # what does not count may hold anything
        c.view(torch.uint8)[~live] = 0x7F
        s[~live] = float("nan")
    dw = torch.full((G, N, K), float("nan"), device=DEV)
    assert dg.dg_grouped_wgrad_fp8_contiguous(p, sp, q, sq, idx, G, dw) is dw
    old = torch.randn(G, N, K, device=DEV).to(BF)
    acc = dg.dg_grouped_wgrad_fp8_contiguous(p, sp, q, sq, idx, G, old.clone(), accumulate=True)
    for i in range(G):
        at = live & (idx == i)
        ops = [t[at] if t.dtype is F else t.view(torch.uint8)[at].view(t.dtype) for t in (p, sp, q, sq)]
        check(dw[i], *ops, what=f"group {i}")
        check(acc[i], *ops, before=old[i], what=f"group {i} accumulated")
        if not at.any():
            assert (dw[i] == 0).all() and torch.equal(acc[i], old[i])


def test_empty():
    z = torch.zeros(0, 256, device=DEV, dtype=torch.uint8)
    s = torch.zeros(0, 2, device=DEV)
    dw = torch.full((256, 256), 5.0, device=DEV)
    assert (dg.dg_wgrad_fp8(z, s, z, s, dw, accumulate=True) == 5).all()
    assert (dg.dg_wgrad_fp8(z, s, z, s, dw) == 0).all()
    idx = torch.zeros(0, device=DEV, dtype=torch.int32)
    assert (dg.dg_grouped_wgrad_fp8_contiguous(z, s, z, s, idx, 3, dtype=BF) == 0).all()
    p, sp, q, sq = make(200, 256, 256)
    none = torch.full((200,), -1, device=DEV, dtype=torch.int32)
    assert (dg.dg_grouped_wgrad_fp8_contiguous(p, sp, q, sq, none, 2) == 0).all()


def test_rows_beyond_two_to_the_31_bytes():
    T, N, K = 140000, 16384, 128
    g = torch.Generator(device=DEV).manual_seed(0)
    p = torch.zeros(T, N, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn)
    last = torch.randint(-4, 5, (200, N), generator=g, device=DEV).float().to(p.dtype)
    p.view(torch.uint8)[T - 200:] = last.view(torch.uint8)
    q = torch.randint(-4, 5, (T, K), generator=g, device=DEV).float().to(p.dtype)
    sp, sq = torch.ones(T, N // 128, device=DEV), torch.ones(T, 1, device=DEV)
    want = last.double().t() @ q[T - 200:].double()
    assert torch.equal(dg.dg_wgrad_fp8(p, sp, q, sq).double(), want)


@pytest.mark.parametrize("T,N,K", [(3000, 128, 256), (300, 1024, 512)])
def test_same_bits_again_graph_and_stream(T, N, K):
    ops = make(T, N, K)
    want = dg.dg_wgrad_fp8(*ops)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dg.dg_wgrad_fp8(*ops, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = dg.dg_wgrad_fp8(*ops)
    for i in range(3):
        ops[1].mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, dg.dg_wgrad_fp8(*ops))


def test_refusals():
    p, sp, q, sq = make(10, 256, 128)
    f = dg.dg_wgrad_fp8
    with pytest.raises(ValueError, match="must be on a GPU"):
        f(p.cpu(), sp, q, sq)
    with pytest.raises(TypeError, match="P must be"):
        f(p.float(), sp, q, sq)
    with pytest.raises(ValueError, match="Q must have shape"):
        f(p, sp, q[:9], sq)
    with pytest.raises(ValueError, match="sP must have shape"):
        f(p, sp[:, :1], q, sq)
    with pytest.raises(ValueError, match="accumulate needs"):
        f(p, sp, q, sq, accumulate=True)
    with pytest.raises(TypeError, match="dW must be"):
        f(p, sp, q, sq, dtype=torch.float16)
    with pytest.raises(ValueError, match="contradicts"):
        f(p, sp, q, sq, torch.zeros(256, 128, device=DEV), dtype=BF)
    with pytest.raises(ValueError, match="contradicts dtype"):
        f(p, sp, q, sq, p_format="e5m2")
    with pytest.raises(dg.DGError, match="SHAPE"):
        f(torch.zeros(10, 200, device=DEV, dtype=torch.uint8), torch.ones(10, 1, device=DEV), q, sq)
    with pytest.raises(dg.DGError, match="SHAPE"):
        dg.dg_grouped_wgrad_fp8_contiguous(p, sp, q, sq, torch.zeros(10, device=DEV, dtype=torch.int32), 0,
                                           torch.zeros(0, 256, 128, device=DEV))
