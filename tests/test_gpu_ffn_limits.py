"""The feed-forward calls at the largest sizes that they take, with whole numbers and scales of powers
of two, so that every sum is exact: the longest K, the widest N, weights and gradients past 2^32 bytes."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import ffn_ref as R  # noqa: E402

DEV = "cuda:0"
BF, E4 = torch.bfloat16, torch.float8_e4m3fn
ACT = 2.0 ** -18                      # the activation's own error (test_gpu_gated.py)


def gen(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    one = torch.tensor([0xB8, 0x00, 0x38], dtype=torch.uint8, device=DEV)         # -1, 0, 1
    codes = lambda *s: one[torch.randint(0, 3, s, generator=g, device=DEV)].view(E4)  # noqa: E731
    scales = lambda *s: torch.exp2(torch.randint(-1, 1, s, generator=g, device=DEV).float())  # noqa: E731
    return codes, scales


def check(H, sH, GU, sGU, gu, what):
    N = gu.shape[1] // 2
    R.check_codes_sharp(GU, sGU, gu, 2.0 ** -23, "e4m3", what)
    h = R.gated(gu[:, :N], gu[:, N:], "silu")
    R.check_codes(H, sH, h, ACT * h.abs(), "e4m3", what)


@pytest.mark.parametrize("M", [1, 64, 130])
def test_gated_longest_k(M):
    N, K = 128, 1 << 22
    codes, scales = gen(M)
    a, b = codes(M, K), codes(2 * N, K)
    # scales 1/2 and 1 of A, 2^-8 of B: a sum of at most 2^22 terms that are multiples of 2^-9, below 2^-8
    sa, sb = scales(M, K // 128), torch.full((2, K // 128), 2.0 ** -8, device=DEV)
    out = dg.dg_gated_fp8_nt(a, sa, b, sb, save=True)
    gu = torch.zeros(M, 2 * N, device=DEV, dtype=torch.float64)
    for k in range(0, K, 1 << 19):
        at = slice(k, k + (1 << 19))
        gu += R.values(a[:, at].contiguous(), sa[:, k // 128:(k >> 7) + 4096]) @ b[:, at].double().t() * 2.0 ** -8
    check(*out, gu, f"{M} rows")


@pytest.mark.parametrize("M", [1, 3, 129])
def test_gated_widest_n(M):
    N, K = 1 << 20, 128
    codes, scales = gen(M)
    a, b, sa, sb = codes(M, K), codes(2 * N, K), scales(M, 1), scales(2 * N // 128, 1)
    sa, sb = sa / 8, sb / 8
    H, sH, GU, sGU = dg.dg_gated_fp8_nt(a, sa, b, sb, save=True)
    gu = R.values(a, sa) @ R.weight_values(b, sb).t()
    check(H, sH, GU, sGU, gu, "widest")
    dh = torch.randint(-3, 4, (M, N), device=DEV).to(BF)
    D, sD = dg.dg_gated_backward(dh, GU, sGU)
    for at in (slice(0, 256), slice(N // 2, N // 2 + 256), slice(N - 256, N)):
        up = slice(N + at.start, N + at.stop)
        blocks, up_blocks = (slice(s.start // 128, s.stop // 128) for s in (at, up))
        part = dg.dg_gated_backward(dh[:, at].contiguous(), torch.cat([GU.view(torch.uint8)[:, s] for s in (at, up)], 1),
                                    torch.cat([sGU[:, s] for s in (blocks, up_blocks)], 1))
        assert torch.equal(torch.cat([D.view(torch.uint8)[:, s] for s in (at, up)], 1), part[0].view(torch.uint8))
        assert torch.equal(torch.cat([sD[:, s] for s in (blocks, up_blocks)], 1), part[1])


@pytest.mark.parametrize("form", ["contiguous", "masked"])
@pytest.mark.parametrize("cap", [40, 200])
def test_gated_groups_past_32_bits(form, cap):
    """The last groups' weights lie more than 2^32 bytes behind the first."""
    G, N, K = 48, 2816, 16384
    codes, scales = gen(cap)
    b = torch.zeros(G, 2 * N, K, dtype=torch.uint8, device=DEV).view(E4)
    sb = torch.full((G, 2 * N // 128, K // 128), 2.0 ** -6, device=DEV)
    used = [0, 46, 47]
    for g in used:
        b[g].view(torch.uint8).copy_(codes(2 * N, K).view(torch.uint8))
    if form == "masked":
        a, sa = codes(G, cap, K), scales(G, cap, K // 128)
        counts = torch.zeros(G, dtype=torch.int32, device=DEV)
        counts[used] = torch.tensor([cap, 7, cap - 1], dtype=torch.int32, device=DEV)
        H, sH, _, _ = dg.dg_grouped_gated_fp8_masked(a, sa, b, sb, counts)
        parts = [(g, a[g, :int(counts[g])], sa[g, :int(counts[g])], H[g, :int(counts[g])], sH[g, :int(counts[g])])
                 for g in used]
    else:
        idx = torch.cat([torch.tensor([g] * cap + [-1] * (-cap % 128), dtype=torch.int32) for g in used]).to(DEV)
        a, sa = codes(idx.numel(), K), scales(idx.numel(), K // 128)
        H, sH, _, _ = dg.dg_grouped_gated_fp8_contiguous(a, sa, b, sb, idx)
        parts = [(g, a[idx == g], sa[idx == g], H[idx == g], sH[idx == g]) for g in used]
    for g, x, s, h, sh in parts:
        gu = R.values(x, s) @ R.weight_values(b[g], sb[g]).t()
        want = R.gated(gu[:, :N], gu[:, N:], "silu")
        R.check_codes(h, sh, want, ACT * want.abs(), "e4m3", f"group {g}")


@pytest.mark.parametrize("turned", [False, True])
def test_widest_weight_gradient(turned):
    T, N, K = 70, 1 << 22, 128
    if turned:
        N, K = K, N
    codes, scales = gen(T)
    p, sp, q, sq = codes(T, N), scales(T, N // 128), codes(T, K), scales(T, K // 128)
    dw = dg.dg_wgrad_fp8(p, sp, q, sq)
    vp, vq = (R.values(c, s).float() for c, s in ((p, sp), (q, sq)))     # whole halves: sums exact in fp32
    assert torch.equal(dw, vp.t() @ vq)


def test_weight_gradients_past_32_bits():
    G, N, K, T = 160, 4096, 4096, 3 * 128 + 50
    codes, scales = gen(0)
    groups = [159, 0, 158, 159]
    idx = torch.tensor([groups[t // 128] for t in range(T)], dtype=torch.int32, device=DEV)
    p, sp, q, sq = codes(T, N), scales(T, N // 128), codes(T, K), scales(T, K // 128)
    dw = torch.full((G, N, K), float("nan"), dtype=BF, device=DEV)
    dg.dg_grouped_wgrad_fp8_contiguous(p, sp, q, sq, idx, G, dw)
    vp, vq = (R.values(c, s).float() for c, s in ((p, sp), (q, sq)))
    for g in (0, 158, 159):
        at = idx == g
        assert torch.equal(dw[g], (vp[at].t() @ vq[at]).to(BF))
    assert all((dw[g] == 0).all() for g in (1, 80, 157))
