"""The norm's backward pass with its gradient in the place of each matrix that it may take."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402

DEV = "cuda:0"


# rows and widths on both sides of the one launch's limits (1024 rows, 8192 columns): there
# workgroups that form the weight's gradient read grad_y and H while others write grad_x
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K", [(1, 128), (5, 7168), (517, 2048), (1024, 1024), (1024, 8192), (1025, 512),
                                 (40, 8320)])
@pytest.mark.parametrize("place", ["grad_y", "grad_h", "H"])
def test_grad_x_in_the_place_of_another(place, T, K, dtype):
    g = torch.Generator(device=DEV).manual_seed(T + K)

    def n(*s):
        return torch.randn(*s, generator=g, device=DEV)

    wide = torch.zeros(3, T, K + 8, device=DEV, dtype=dtype)          # rows apart, the rest stays
    grad_y, grad_h, H = (m[:, :K] for m in wide)
    for m in (grad_y, grad_h, H):
        m.copy_(n(T, K))
    w = 1 + 0.1 * n(K)
    rstd = dg.dg_rms_norm_fp8(H, w, codes=False, save=True)[4]
    want = dg.dg_rms_norm_backward(grad_y, H, rstd, w, grad_h=grad_h)
    for _ in range(3):
        mine = dict(zip(("grad_y", "grad_h", "H"), (m[:, :K] for m in wide.clone())))
        got = dg.dg_rms_norm_backward(mine["grad_y"], mine["H"], rstd, w, grad_h=mine["grad_h"], grad_x=mine[place])
        assert got[0] is mine[place]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for name, m in mine.items():
            if name != place:
                assert torch.equal(m, dict(grad_y=grad_y, grad_h=grad_h, H=H)[name])
    assert (wide[:, :, K:] == 0).all()
