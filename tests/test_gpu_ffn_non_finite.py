"""NaN and infinities that reach the feed-forward block through its weights or its gradients show in
what it returns: the block's quantisation of them is the package's own call."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16
BAD = [float("nan"), float("inf"), -float("inf")]


def make():
    g = torch.Generator(device=DEV).manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return n(40, 256).to(BF), n(256, 256) / 16, n(256, 128) / 11, n(40, 256).to(BF)


@pytest.mark.parametrize("bad", BAD)
def test_in_the_gradient(bad):
    x, w13, w2, go = make()
    leaves = [t.requires_grad_() for t in (x, w13, w2)]
    want = torch.autograd.grad(dg.gated_ffn(*leaves)[0], leaves, go)
    go[7, 30] = bad
    dx, d13, d2 = torch.autograd.grad(dg.gated_ffn(*leaves)[0], leaves, go)
    assert not dx[7].isfinite().any()                    # the row's
    assert torch.equal(dx[:7], want[0][:7]) and torch.equal(dx[8:], want[0][8:])
    assert not d2[30].isfinite().any() and not d13.isfinite().all()
    assert torch.equal(d2[128:], want[2][128:])          # other blocks of its row


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("which", [0, 1])
def test_in_a_weight(which, bad):
    x, w13, w2, _ = make()
    (w13, w2)[which][3, 20] = bad
    out, _ = dg.gated_ffn(x, w13, w2)
    assert not out[:, 3].isfinite().any()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("bad", BAD)
def test_a_block_is_not_finite(bad, dtype, fmt):
    """Of the quantisation's own: the block's values are NaN or infinite, the others as they were."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(300, 512, generator=g, device=DEV).to(dtype)
    calls = {"row": dg.dg_quantize_fp8_1x128, "square": dg.dg_quantize_fp8_128x128}
    want = {k: f(x, fmt) for k, f in calls.items()}
    x[200, 300] = bad
    for k, f in calls.items():
        q, s = f(x, fmt)
        rows = slice(200, 201) if k == "row" else slice(128, 256)
        at = (200 if k == "row" else 1, 2)
        assert not s[at].isfinite()
        q0, s0 = want[k]
        s[at] = s0[at]
        assert torch.equal(s, s0)
        a, b = q.view(torch.uint8).clone(), q0.view(torch.uint8)
        a[rows, 256:384] = b[rows, 256:384]
        assert torch.equal(a, b)
