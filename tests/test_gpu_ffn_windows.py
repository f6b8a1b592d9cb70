"""Feed-forward calls past what one look or launch takes, in value: weight gradients of groups whose
rows lie in several windows of 256 blocks, norms whose offsets pass 32 bits, exact workspaces of the
norm's backward pass in two launches."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import ffn_ref as R  # noqa: E402

DEV = "cuda:0"
BF, F = torch.bfloat16, torch.float32


def exact_operands(T, N, K, seed):
    """Codes that are small whole numbers and scales of powers of two: every product and, of up to
    2^17 rows, every sum is exact."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def whole(*s):
        return torch.randint(-3, 4, s, generator=g, device=DEV).float().to(torch.float8_e4m3fn)

    def power(*s):
        return torch.exp2(torch.randint(-1, 2, s, generator=g, device=DEV).float())

    return whole(T, N), power(T, N // 128), whole(T, K), power(T, K // 128)


def block_groups(layout, blocks):
    b = torch.arange(blocks)
    if layout == "late":              # group 1 only behind the first window, group 2 in the third
        return torch.where(b >= 515, 2, torch.where(b >= 300, 1, 0))
    if layout == "apart":             # group 0 at both ends: a whole window without it between
        return torch.where((b < 3) | (b >= 590), 0, 1 + b % 2)
    if layout == "holes":             # and windows of rows that count nowhere
        return torch.where((b > 40) & (b < 560), -1, b % 3)
    return b % 3                      # over all of them


@pytest.mark.parametrize("tail", [0, 1, 77])
@pytest.mark.parametrize("layout", ["late", "apart", "holes", "over"])
@pytest.mark.parametrize("G,N,K", [(3, 128, 128), (3, 128, 256), (150, 128, 256)])
def test_grouped_weight_gradients_over_many_blocks(G, N, K, layout, tail):
    """Three groups of the many have rows; their sums are split where the tiles are few."""
    blocks = 600
    idx = block_groups(layout, blocks).repeat_interleave(128).int().to(DEV)
    if tail:
        idx = torch.cat([idx, torch.full((tail,), 2, dtype=torch.int32, device=DEV)])
    idx[5:9] = -1                     # rows that do not count, inside a block
    T = idx.numel()
    split = dg.dg_wgrad_workspace_bytes(T, N, K, G) > 0
    assert split == (G == 3)
    p, sp, q, sq = exact_operands(T, N, K, tail + K)
    live = R.written(idx, G)
    sp[~live] = float("nan")
    got = dg.dg_grouped_wgrad_fp8_contiguous(p, sp, q, sq, idx, G)
    for i in range(G):
        if i < 3:
            at = (live & (idx == i)).nonzero()[:, 0]
            vp, vq = (R.values(c.view(torch.uint8)[at].view(c.dtype), s[at]) for c, s in ((p, sp), (q, sq)))
            assert torch.equal(got[i].double(), vp.t() @ vq)
        else:
            assert (got[i] == 0).all()


def test_norm_past_32_bits_in_value():
    """Rows 4096 apart, 2^20 + 5 of them: offsets past 2^32 bytes, and of the forward pass a second
    launch.  Every row of either pass against the same rows in calls of a few thousand."""
    T, K, wide = (1 << 20) + 5, 128, 4096
    g = torch.Generator(device=DEV).manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    far = lambda: torch.empty(T, wide, device=DEV, dtype=BF)[:, :K]  # noqa: E731
    x, dy, gx = far(), far(), far()
    x.copy_(n(T, K))
    dy.copy_(n(T, K))
    gx.fill_(-77.0)
    gh, w = n(T, K).to(BF), 1 + 0.1 * n(K)
    q, s, _, y, rstd = dg.dg_rms_norm_fp8(x, w, bf16=True, save=True)
    dx, dw = dg.dg_rms_norm_backward(dy, x, rstd, w, grad_h=gh, grad_x=gx)
    step = (1 << 17) + 1                                 # eight calls, the last one as large as the others
    for at in range(0, T, step):
        rows = slice(at, min(at + step, T))
        a, b = x[rows].contiguous(), dy[rows].contiguous()
        part = dg.dg_rms_norm_fp8(a, w, bf16=True, save=True)
        assert torch.equal(q[rows].view(torch.uint8), part[0].view(torch.uint8)) and torch.equal(s[rows], part[1])
        assert torch.equal(y[rows], part[3]) and torch.equal(rstd[rows], part[4])
        assert torch.equal(dx[rows], dg.dg_rms_norm_backward(b, a, part[4], w, grad_h=gh[rows])[0])
    for at in (slice(0, 64), slice(T - 64, T)):          # and some of them against the formula
        want, _, mag, _ = R.norm_backward(dy[at], x[at], rstd[at], w, gh[at])
        assert ((dx[at].double() - want).abs() <= R.HALF[BF] * 1.01 * want.abs() + 100 * 2.0 ** -24 * mag).all()
    want_w, mag_w = torch.zeros(2, K, device=DEV, dtype=torch.float64)
    for at in range(0, T, step):
        rows = slice(at, min(at + step, T))
        _, a, _, b = R.norm_backward(dy[rows], x[rows], rstd[rows], w)
        want_w += a
        mag_w += b
    assert ((dw.double() - want_w).abs() <= (T + 4) * 2.0 ** -24 * mag_w).all()
    # such errors have either sign: 512 workgroups add 2048 rows each
    assert ((dw.double() - want_w).abs() <= 2100 * 2.0 ** -24 * mag_w).all()


@pytest.mark.parametrize("T,K", [(1025, 128), (3000, 384), (5, 8320), (700, 16384)])
def test_norm_backward_workspace_of_two_launches(T, K):
    g = torch.Generator(device=DEV).manual_seed(T)
    x, dy, w = (torch.randn(*s, generator=g, device=DEV) for s in ((T, K), (T, K), (K,)))
    rstd = dg.dg_rms_norm_fp8(x, w, codes=False, save=True)[4]
    need = dg.dg_rms_norm_backward_workspace_bytes(T, K)
    whole = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=DEV)
    got = dg.dg_rms_norm_backward(dy, x, rstd, w, workspace=whole[256:256 + need])
    assert (whole[:256] == 0xFF).all() and (whole[-256:] == 0xFF).all()
    assert (whole[256:-256] != 0xFF).any()                # it is used
    want = dg.dg_rms_norm_backward(dy, x, rstd, w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
