"""The stack of feed-forward layers of examples/feed_forward.py: it runs, and its gradients are
those of the same stack in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

from examples import feed_forward  # noqa: E402
from tests import ffn_ref as R  # noqa: E402


def test_runs():
    feed_forward.main()


def test_gradients():
    T, K, N = 300, 256, 384
    stack = feed_forward.Stack(2, K, N)
    g = torch.Generator(device="cuda:0").manual_seed(3)
    x = torch.randn(T, K, generator=g, device="cuda:0").bfloat16().requires_grad_()
    go = torch.randn(T, K, generator=g, device="cuda:0").bfloat16()
    out = stack(x)
    out.backward(go)
    leaves = [x] + list(stack.parameters())
    exact = [v.detach().double().requires_grad_() for v in leaves]
    a, h, rest = exact[0], None, exact[1:]
    for i in range(2):
        w, w13, w2 = rest[3 * i:3 * i + 3]
        h = a if h is None else h + a
        gu = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w @ w13.t()
        a = R.gated(gu[:, :N], gu[:, N:], "silu") @ w2.t()
    want = a + h
    grads = torch.autograd.grad((want * go.double()).sum(), exact)
    rel = lambda p, q: float((p.detach().double() - q.detach()).norm() / q.detach().norm())  # noqa: E731
    # A code of a normal binade is off by 2^-4 / sqrt(3) of its value at most.  One layer's output
    # holds 6 such errors and its gradients 9 (its own codes, the checkpoint's, the incoming
    # gradient's), each independent; the second layer's input holds the first's 6, the first's
    # incoming gradient the second's 9.
    assert rel(out, want) < 12 ** 0.5 * 0.0361
    for leaf, grad in zip(leaves, grads):
        assert leaf.grad.shape == leaf.shape and rel(leaf.grad, grad) < 24 ** 0.5 * 0.0361
