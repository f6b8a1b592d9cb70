"""The feed-forward operators together, as a program uses them: gated_ffn against the block in 64
bits with the roundings to 8 bits that the calls make, decode steps, and a captured step."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import ffn_ref as R  # noqa: E402

DEV = "cuda:0"
BF, F = torch.bfloat16, torch.float32


def make(T, K, N, M, dtype=BF, seed=0, residual=True):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=g, device=DEV)

    x = n(T, K).to(dtype).requires_grad_()
    r = (2 * n(T, K)).to(dtype).requires_grad_() if residual else None
    w = (1 + 0.2 * n(K)).requires_grad_()
    w13 = (n(2 * N, K) * K ** -0.5).requires_grad_()
    w2 = (n(M, N) * N ** -0.5).to(BF).requires_grad_()
    return x, r, w, w13, w2, n


def exact(x, r, w, w13, w2, act, go, gh):
    """The block and its gradients in 64 bits without any rounding."""
    leaves = [v.detach().double().requires_grad_() for v in (x, r, w, w13, w2) if v is not None]
    x64, r64 = leaves[0], leaves[1] if r is not None else None
    w64, a, b = leaves[-3:]
    h = x64 if r64 is None else x64 + r64
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w64
    gu = y @ a.t()
    N = a.shape[0] // 2
    out = R.gated(gu[:, :N], gu[:, N:], act) @ b.t()
    total = (out * go.double()).sum() + (0 if gh is None else (h * gh.double()).sum())
    return out, h, torch.autograd.grad(total, leaves)


def rel(a, b):
    return float((a.detach().double() - b.detach()).norm() / b.detach().norm())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,K,N,M,dtype,residual", [(1, 256, 128, 256, BF, True), (77, 512, 384, 512, BF, True),
                                                   (300, 1024, 640, 256, F, False), (1000, 768, 1024, 768, BF, True)])
def test_gated_ffn(T, K, N, M, dtype, residual, act):
    x, r, w, w13, w2, n = make(T, K, N, M, dtype, T, residual)
    out, h = dg.gated_ffn(x, w13, w2, residual=r, norm_weight=w, activation=act)
    go, gh = n(T, M).to(BF), (n(T, K).to(dtype) if residual else None)
    assert out.dtype is BF and (h is None) == (not residual)
    torch.autograd.backward([out] + ([h] if residual else []), [go] + ([gh] if residual else []))
    want, want_h, grads = exact(x, r, w, w13, w2, act, go, gh)
    # A code of a normal binade is off by a uniform part of a step: 2^-4 / sqrt(3) of its value
    # at most, 0.036.  The output's terms hold codes of y, of both projections' weights (twice,
    # for gate and up), of h and of the down projection's weight: 6 such errors, and the
    # gradients' besides those of G and U and the incoming gradient's up to 9, each independent
    # from element to element: sqrt(9) 0.036.
    assert rel(out, want) < 6 ** 0.5 * 0.0361
    if residual:
        assert torch.equal(h, (x.float() + r.float()).to(dtype))
    leaves = [v for v in (x, r, w, w13, w2) if v is not None]
    for leaf, g in zip(leaves, grads):
        assert leaf.grad.dtype is leaf.dtype and leaf.grad.shape == leaf.shape
        assert rel(leaf.grad, g) < 9 ** 0.5 * 0.0361
    if residual:
        assert torch.equal(x.grad, r.grad)


def test_gated_ffn_is_its_calls():
    """The function's gradients are bit for bit what its calls give one after another."""
    T, K, N, M = 200, 512, 256, 384
    x, r, w, w13, w2, n = make(T, K, N, M)
    go, gh = n(T, M).to(BF), n(T, K).to(BF)
    out, h = dg.gated_ffn(x, w13, w2, residual=r, norm_weight=w)
    torch.autograd.backward([out, h], [go, gh])
    with torch.no_grad():
        b13, s13 = dg.dg_quantize_fp8_128x128(w13)
        b2, s2 = dg.dg_quantize_fp8_128x128(w2)
        q, s, h2, _, rstd = dg.dg_rms_norm_fp8(x, w, residual=r, save=True)
        a, sa, gu, sgu = dg.dg_gated_fp8_nt(q, s, b13, s13, save=True)
        assert torch.equal(out, dg.dg_gemm_fp8_nt(a, sa, b2, s2)) and torch.equal(h, h2)
        d, sd = dg.dg_quantize_fp8_1x128(go)
        da = dg.dg_gemm_fp8_nt(d, sd, dg.dg_transpose_fp8(b2), s2.t().contiguous())
        assert torch.equal(w2.grad, dg.dg_wgrad_fp8(d, sd, a, sa, dtype=BF))
        d, sd = dg.dg_gated_backward(da, gu, sgu)
        assert torch.equal(w13.grad, dg.dg_wgrad_fp8(d, sd, q, s))
        dy = dg.dg_gemm_fp8_nt(d, sd, dg.dg_transpose_fp8(b13), s13.t().contiguous())
        dx, dw = dg.dg_rms_norm_backward(dy, h2, rstd, w, grad_h=gh)
        assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw)


def test_parts_of_the_gradient():
    """Leaves that need none get none; a loss on one output only; once differentiable."""
    x, r, w, w13, w2, n = make(40, 256, 128, 256)
    out, h = dg.gated_ffn(x.detach(), w13, w2.detach(), residual=r.detach(), norm_weight=w.detach())
    (g,) = torch.autograd.grad(out.float().sum(), [w13])
    assert g.shape == w13.shape
    out, h = dg.gated_ffn(x, w13, w2, residual=r, norm_weight=w)
    gx, gr = torch.autograd.grad(h.float().sum(), [x, r])
    assert (gx == 1).all() and (gr == 1).all()
    out, h = dg.gated_ffn(x, w13, w2)
    assert h is None
    (g,) = torch.autograd.grad(out.float().square().sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_empty_batch():
    x, _, w, w13, w2, _ = make(0, 256, 128, 256, residual=False)
    out, _ = dg.gated_ffn(x, w13, w2, norm_weight=w)
    out.float().sum().backward()
    assert out.shape == (0, 256) and (w13.grad == 0).all() and (w2.grad == 0).all() and (w.grad == 0).all()


def test_decode_steps_in_a_graph():
    """norm, gated block and down projection of a few tokens, dense and through masked experts,
    captured once and replayed on new tokens and counts, with eager work between."""
    T, K, N, E = 24, 512, 256, 4
    x, r, w, w13, w2, n = make(T, K, N, K)
    with torch.no_grad():
        b13, b2 = dg.dg_quantize_fp8_128x128(w13), dg.dg_quantize_fp8_128x128(w2)
        e13 = [dg.dg_quantize_fp8_128x128(n(2 * N, K)) for _ in range(E)]
        e13 = torch.stack([q.view(torch.uint8) for q, _ in e13]), torch.stack([s for _, s in e13])
        x, r = x.detach(), r.detach()
        counts = torch.tensor([3, 0, 24, 9], device=DEV, dtype=torch.int32)

        def step():
            q, s, h, y, _ = dg.dg_rms_norm_fp8(x, w.detach(), residual=r, bf16=True)
            a, sa, _, _ = dg.dg_gated_fp8_nt(q, s, *b13)
            out = dg.dg_gemm_fp8_nt(a, sa, *b2)
            ea = q.view(torch.uint8).expand(E, T, K).contiguous(), s.expand(E, T, K // 128).contiguous()
            eh, es, _, _ = dg.dg_grouped_gated_fp8_masked(*ea, *e13, counts)
            return out, h, y, eh.view(torch.uint8), es

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        for i in range(4):
            x.copy_(n(T, K))
            counts.copy_(torch.randint(0, T + 1, (E,), device=DEV))
            want = step()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(held, want):
                assert torch.equal(a, b)


def test_two_streams_at_once():
    """The same calls on two streams, each with its own kept workspaces."""
    jobs = []
    for i in range(2):
        x, r, w, w13, w2, n = make(60 + 500 * i, 1024, 512, 256, seed=i)
        go = n(x.shape[0], 256).to(BF)
        out, h = dg.gated_ffn(x, w13, w2, residual=r, norm_weight=w)
        want = (out, h) + torch.autograd.grad([out], [x, w, w13, w2], [go])
        jobs.append((x, r, w, w13, w2, go, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, (x, r, w, w13, w2, go, _, stream) in enumerate(jobs):
            with torch.cuda.stream(stream):
                out, h = dg.gated_ffn(x, w13, w2, residual=r, norm_weight=w)
                got[k].append((out, h) + torch.autograd.grad([out], [x, w, w13, w2], [go]))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            for a, b in zip(run, jobs[k][6]):
                assert torch.equal(a, b)
