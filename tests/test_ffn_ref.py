"""The 64-bit forms that the feed-forward operators are tested against: their gradients
against differences and autograd, their quantisation against the oracle's."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from tests import ffn_ref as R  # noqa: E402


def _differences(f, x, d, h=1e-5):
    return float((f(x + h * d) - f(x - h * d)).sum()) / (2 * h)


@pytest.mark.parametrize("weight", [False, True])
def test_norm_gradient(weight):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(3, 128, generator=g, dtype=torch.float64)
    w = torch.rand(128, generator=g, dtype=torch.float64) + 0.5 if weight else None
    dy = torch.randn(3, 128, generator=g, dtype=torch.float64)
    _, rstd, _ = R.norm(x, w)
    dx, dw, mag, _ = R.norm_backward(dy, x, rstd, w)
    assert (dx.abs() <= mag * (1 + 1e-12)).all()
    for i in range(4):
        d = torch.randn(3, 128, generator=g, dtype=torch.float64)
        # a central difference of step h is off by h^2 times a third derivative of order 1
        want = _differences(lambda v: R.norm(v, w)[2] * dy, x, d)
        assert abs(want - float((dx * d).sum())) < 1e-6 * max(1.0, abs(want))
        if weight:
            dd = d[0]
            want = _differences(lambda v: R.norm(x, v)[2] * dy, w, dd)
            assert abs(want - float((dw * dd).sum())) < 1e-6 * max(1.0, abs(want))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_gradient(act):
    g = torch.Generator().manual_seed(1)
    gu = 2 * torch.randn(5, 16, generator=g, dtype=torch.float64)
    dh = torch.randn(5, 8, generator=g, dtype=torch.float64)
    want = R.gated_backward(dh, gu[:, :8], gu[:, 8:], act)
    leaf = gu.clone().requires_grad_()
    lib = torch.nn.functional.silu if act == "silu" else lambda v: torch.nn.functional.gelu(v, approximate="tanh")
    (auto,) = torch.autograd.grad(lib(leaf[:, :8]) * leaf[:, 8:], leaf, dh)
    assert torch.allclose(want, auto, rtol=1e-12, atol=1e-14)
    d = torch.randn(5, 16, generator=g, dtype=torch.float64)
    diff = _differences(lambda v: R.gated(v[:, :8], v[:, 8:], act) * dh, gu, d)
    assert abs(diff - float((want * d).sum())) < 1e-6 * max(1.0, abs(diff))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantisation_is_the_oracles(fmt):
    x = np.random.default_rng(2).standard_normal((7, 384)).astype(np.float32)
    x[2, 128:256] = 0
    q, s = R.quantise(torch.from_numpy(x), fmt)
    q_ref, s_ref = oracle.quantize_1x128(x, fmt)
    assert np.array_equal(q.view(torch.uint8).numpy(), q_ref) and np.array_equal(s.numpy(), s_ref)
    R.check_codes(q, s, torch.from_numpy(x).double(), 0.0, fmt)
    R.check_codes_sharp(q, s, torch.from_numpy(x).double(), 2.0 ** -22, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_the_checks_see_mistakes(fmt):
    """A code one step off, a scale of the next block, a value a little off."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(4, 256, generator=g)
    q, s = R.quantise(x, fmt)
    v = x.double()
    worse = q.clone()
    worse.view(torch.uint8)[1, 5] ^= 1
    for bad in ((worse, s), (q, s.flip(1)), (q, s * 1.001)):
        with pytest.raises(AssertionError):
            R.check_codes(*bad, v, 1e-7, fmt)
    with pytest.raises(AssertionError):
        R.check_codes_sharp(worse, s, v, 1e-6, fmt)
    # a thousandth of the values' size shows in some codes
    q2, s2 = R.quantise(x * 1.02, fmt)
    with pytest.raises(AssertionError):
        R.check_codes(q2, s2, v, 1e-7, fmt)


def test_rows_that_are_written():
    idx = torch.tensor([0] * 100 + [-1] * 28 + [5] * 3 + [0] * 125 + [1] * 7, dtype=torch.int32)
    w = R.written(idx, 5)
    assert w[:100].all() and not w[100:256].any() and w[256:].all()
