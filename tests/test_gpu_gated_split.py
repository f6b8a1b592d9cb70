"""The gated block where its few tiles are split over the GPU (sums of pieces, joined by a second
kernel) against the formulas in 64 bits: masked counts of every kind, dense rows on both sides of
each tile, every pair of formats, in a workspace of just the size that is asked for."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import ffn_ref as R  # noqa: E402
from tests.test_gpu_gated import FORMATS, check, gen, weights  # noqa: E402

DEV = "cuda:0"

# check()'s bound counts 128 + 3 + K / 128 roundings of a sum.  Here a path has 128 at most inside
# a K block, one for the scales' product, those of its piece's blocks and, joined, one for each
# second piece and one more: pieces have four blocks or more, so that is less than before.


def workspace(kind, rows, N, K, G=1):
    """A workspace of just the size asked for, of NaN, between bytes that no call may touch."""
    need = dg.dg_gated_workspace_bytes(kind, rows, N, K, G)
    assert need > 0, "not split any more: another size for this test"
    whole = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=DEV)
    return whole, whole[256:256 + need]


def untouched(whole):
    return bool((whole[:256] == 0xFF).all() and (whole[-256:] == 0xFF).all())


MASKED = [(1, 1, 256, 2048, [1]), (3, 16, 256, 2048, [16, 0, 5]), (4, 64, 256, 2176, [0, 64, 33, 1]),
          (3, 40, 384, 4096, [-5, 99, 40]), (64, 20, 256, 2048, list(range(-22, 42))),
          (5, 128, 256, 2048, [128, 0, 127, 3, 64]), (2, 100, 640, 2560, [99, 100]),
          (3, 200, 256, 2048, [200, 129, 128]), (2, 513, 128, 2048, [513, 257]), (4, 300, 256, 2176, [0, 0, 0, 0]),
          (4, 300, 256, 4096, [300, -1, 1, 400]), (64, 130, 128, 4096, [(7 * i) % 140 - 5 for i in range(64)])]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("case", range(len(MASKED)))
def test_masked(case, act):
    G, cap, N, K, counts = MASKED[case]
    fa, fb, fmt = FORMATS[(case + (act == "gelu")) % 4]
    g, n = gen(case)
    a, sa = R.quantise(n(G, cap, K), fa)
    b, sb = weights(n, K, N, G, fb)
    rows = [max(0, min(c, cap)) for c in counts]
    live = torch.arange(cap, device=DEV) < torch.tensor(rows, device=DEV)[:, None]
    a.view(torch.uint8)[~live] = 0x7F                # NaN in either format
    sa[~live] = float("nan")
    H = torch.full((G, cap, N), 0x55, dtype=torch.uint8, device=DEV)
    sH = torch.full((G, cap, N // 128), -7.0, device=DEV)
    mm = torch.tensor(counts, dtype=torch.int32, device=DEV)
    whole, ws = workspace(dg.DG_MASKED, cap, N, K, G)
    run = lambda ws: dg.dg_grouped_gated_fp8_masked(a, sa, b, sb, mm, H, sH, activation=act, fmt=fmt,  # noqa: E731
                                                    workspace=ws)
    out = run(ws)
    assert untouched(whole) and (H[~live] == 0x55).all() and (sH[~live] == -7).all()
    for i, r in enumerate(rows):
        if r:
            check(out[0][i, :r], out[1][i, :r], None, None, R.values(a[i, :r], sa[i, :r]),
                  R.weight_values(b[i], sb[i]), act, fmt, f"group {i} {fa} {fb} {fmt}")
    with pytest.raises(dg.DGError, match="WORKSPACE"):
        run(ws[:-16])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 256, 2048), (33, 384, 2176), (64, 2048, 2048), (65, 256, 2048),
                                   (100, 1152, 2048), (128, 128, 7168), (129, 256, 2176), (200, 640, 2048),
                                   (255, 384, 2560), (300, 512, 2048), (1000, 256, 4096)])
def test_dense(M, N, K, save, act):
    fa, fb, fmt = FORMATS[(M + N // 128 + save + 2 * (act == "gelu")) % 4]
    g, n = gen(M + N + K)
    a, sa = R.quantise(n(M, K), fa)
    b, sb = weights(n, K, N, fmt=fb)
    whole, ws = workspace(dg.DG_DENSE, M, N, K)
    out = dg.dg_gated_fp8_nt(a, sa, b, sb, activation=act, fmt=fmt, save=save, workspace=ws)
    assert untouched(whole) and (out[2] is None) == (not save)
    check(*out, R.values(a, sa), R.weight_values(b, sb), act, fmt, f"{M}x{N}x{K} {fa} {fb} {fmt}")
    with pytest.raises(dg.DGError, match="WORKSPACE"):
        dg.dg_gated_fp8_nt(a, sa, b, sb, activation=act, fmt=fmt, save=save, workspace=ws[:-16])


@pytest.mark.parametrize("fa,fb,fmt", FORMATS)
@pytest.mark.parametrize("M", [40, 90, 200])
def test_formats(M, fa, fb, fmt):
    """Both tile heights with each pair of operand formats."""
    g, n = gen(M)
    a, sa = R.quantise(n(M, 2304), fa)
    b, sb = weights(n, 2304, 384, fmt=fb)
    whole, ws = workspace(dg.DG_DENSE, M, 384, 2304)
    out = dg.dg_gated_fp8_nt(a, sa, b, sb, fmt=fmt, save=True, workspace=ws)
    assert untouched(whole)
    check(*out, R.values(a, sa), R.weight_values(b, sb), "silu", fmt, f"{fa} {fb} {fmt}")


@pytest.mark.parametrize("M", [5, 64, 100, 300])
def test_whole_numbers(M):
    """Exact projections: every code of gate and up is the one of the value."""
    g, n = gen(9)
    K, N = 2048, 256
    a = torch.randint(-3, 4, (M, K), generator=g, device=DEV).float()
    b = torch.randint(-2, 3, (2 * N, K), generator=g, device=DEV).float()
    sa = torch.exp2(torch.randint(-6, -3, (M, K // 128), generator=g, device=DEV).float())
    sb = torch.exp2(torch.randint(-3, 0, (2 * N // 128, K // 128), generator=g, device=DEV).float())
    a, b = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
    assert dg.dg_gated_workspace_bytes(dg.DG_DENSE, M, N, K) > 0
    _, _, GU, sGU = dg.dg_gated_fp8_nt(a, sa, b, sb, save=True)
    gu = R.values(a, sa) @ R.weight_values(b, sb).t()
    R.check_codes_sharp(GU, sGU, gu, 2.0 ** -23, "e4m3", "gate and up")
