"""A layer of experts trained through the calls, as a program chains them: norm, gated block and down
projection in the contiguous form, their backward passes and the weight gradients of each expert,
against the layer in 64 bits, each call against 64 bits on what it was given, and captured."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import ffn_ref as R  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16
E, CHOICES = 5, 2


def bytes_of(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


def experts(weights):
    """Codes and 128x128 scales of E matrices, and of their transposes."""
    pairs = [dg.dg_quantize_fp8_128x128(w) for w in weights]
    turned = [(dg.dg_transpose_fp8(q), s.t()) for q, s in pairs]
    return tuple((torch.stack([bytes_of(q) for q, _ in p]).view(torch.float8_e4m3fn), torch.stack([s for _, s in p]))
                 for p in (pairs, turned))


def layout(ids, rows):
    """Of T x CHOICES expert ids: each choice's row in the contiguous form and the rows' groups, without
    readback; rows that are no choice's belong to no group."""
    flat = ids.reshape(-1)
    counts = (flat[:, None] == torch.arange(E, device=DEV)).sum(0)
    ends = ((counts + 127) // 128 * 128).cumsum(0)
    first = ends - (counts + 127) // 128 * 128
    place = ((flat[:, None] == flat[None]) & torch.ones(len(flat), len(flat), dtype=torch.bool, device=DEV).tril(-1)).sum(1)
    at = first[flat] + place
    group = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    group[at] = flat.int()
    return at, group


class Layer:
    def __init__(self, T, K, N, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.n = lambda *s: torch.randn(*s, generator=g, device=DEV)
        n = self.n
        self.T, self.K, self.N = T, K, N
        self.rows = -(-T * CHOICES // 128) * 128 + 128 * E
        self.x, self.r, self.go, self.gh = (n(T, K).to(BF) for _ in range(4))
        self.w = 1 + 0.2 * n(K)
        self.w13, self.w2 = n(E, 2 * N, K) * K ** -0.5, n(E, K, N) * N ** -0.5
        self.p = torch.rand(T, CHOICES, generator=g, device=DEV) + 0.5
        self.choose(g)
        self.g = g

    def choose(self, g, least=0):
        """Two experts of each token, none of them the first `least`."""
        self.ids = torch.rand(self.T, E - least, generator=g, device=DEV).argsort(1)[:, :CHOICES] + least

    def step(self, act="silu"):
        (b13, s13), (t13, st13) = experts(self.w13)
        (b2, s2), (t2, st2) = experts(self.w2)
        at, group = layout(self.ids, self.rows)
        token = torch.arange(self.T, device=DEV).repeat_interleave(CHOICES)
        q, s, h, _, rstd = dg.dg_rms_norm_fp8(self.x, self.w, residual=self.r, save=True)
        # rows of no choice hold NaN wherever a program may leave anything
        qc = torch.full((self.rows, self.K), 0x7F, dtype=torch.uint8, device=DEV)
        sc = torch.full((self.rows, self.K // 128), float("nan"), device=DEV)
        qc[at], sc[at] = q.view(torch.uint8)[token], s[token]
        qc = qc.view(q.dtype)
        a, sa, gu, sgu = dg.dg_grouped_gated_fp8_contiguous(qc, sc, b13, s13, group, activation=act, save=True)
        c = dg.dg_grouped_gemm_fp8_contiguous(a, sa, b2, s2, group)
        p = self.p.view(-1, 1)
        out = (p * c[at].float()).view(self.T, CHOICES, self.K).sum(1)
        dc = torch.zeros(self.rows, self.K, dtype=BF, device=DEV)
        dc[at] = (p * self.go[token].float()).to(BF)
        d, sd = dg.dg_quantize_fp8_1x128(dc)
        sd.masked_fill_((group < 0)[:, None], float("nan"))
        da = dg.dg_grouped_gemm_fp8_contiguous(d, sd, t2, st2, group)
        dw2 = dg.dg_grouped_wgrad_fp8_contiguous(d, sd, a, sa, group, E)
        D, sD = dg.dg_gated_backward(da, gu, sgu, group_idx=group, groups=E, activation=act)
        dw13 = dg.dg_grouped_wgrad_fp8_contiguous(D, sD, qc, sc, group, E, dtype=BF)
        dq = dg.dg_grouped_gemm_fp8_contiguous(D, sD, t13, st13, group)
        dy = dq[at].float().view(self.T, CHOICES, self.K).sum(1).to(BF)
        dx, dw = dg.dg_rms_norm_backward(dy, h, rstd, self.w, grad_h=self.gh)
        self.held = dict(at=at, group=group, qc=qc, sc=sc, a=a, sa=sa, gu=gu, sgu=sgu, d=d, sd=sd, da=da, D=D, sD=sD)
        return out, h, dx, dw, dw13, dw2

    def exact(self, act):
        """Outputs and gradients in 64 bits, without any rounding."""
        leaves = [v.double().requires_grad_() for v in (self.x, self.r, self.w, self.w13, self.w2)]
        x, r, w, w13, w2 = leaves
        h = x + r
        y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w
        out = 0
        for j in range(CHOICES):
            for e in range(E):
                gu = y @ w13[e].t()
                c = R.gated(gu[:, :self.N], gu[:, self.N:], act) @ w2[e].t()
                out = out + torch.where(self.ids[:, j:j + 1] == e, self.p[:, j:j + 1].double() * c, 0.0)
        total = (out * self.go.double()).sum() + (h * self.gh.double()).sum()
        gx, _, gw, g13, g2 = torch.autograd.grad(total, leaves)
        return out, h, gx, gw, g13, g2


def rel(a, b):
    return float((a.double() - b.detach()).norm() / b.detach().norm())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,K,N", [(1, 256, 128), (60, 512, 256), (333, 768, 640), (1000, 512, 384)])
def test_training_step(T, K, N, act):
    m = Layer(T, K, N, T)
    if T == 333:
        m.choose(m.g, least=1)                       # an expert without rows
    got = m.step(act)
    want = m.exact(act)
    # codes are off by 2^-4 / sqrt(3) of themselves at most, uniformly and each on its own: an
    # output's terms hold 6 of them, a gradient's 9 at most (the dense layer's); a norm of
    # independent choices' sums grows as their errors' does
    for i, (a, b) in enumerate(zip(got, want)):
        assert a.shape == b.shape
        assert rel(a, b) < (2.0 ** -8 if i == 1 else (6 if i == 0 else 9) ** 0.5 * 0.0361), i
    for e in range(E):
        if not (m.ids == e).any():
            assert (got[4][e] == 0).all() and (got[5][e] == 0).all()
    # each call on what it was given
    v = m.held
    live = v["group"] >= 0
    assert int(live.sum()) == T * CHOICES and torch.equal(R.written(v["group"], E), live)
    g, u = R.values(v["gu"][live], v["sgu"][live]).chunk(2, 1)
    dh = v["da"][live].double()
    d = R.gated_backward(dh, g, u, act)
    # the sigmoid to 2^-18; the derivative's two parts may cancel, so its error goes by their sum, and
    # near 1, 1 - s is off by the error of s itself: |g dz| (2^-22) beside it
    s, dz = R.sigmoid_of(g, act)
    mag = torch.cat([(dh * u).abs() * (s + (g * s * (1 - s) * dz).abs() + 2.0 ** -4 * (g * s * dz).abs()),
                     (dh * g * s).abs()], 1)
    R.check_codes(v["D"][live], v["sD"][live], d, 2.0 ** -18 * mag, "e4m3", "D")
    for dw, (p, sp), (q, sq) in ((got[4], (v["D"], v["sD"]), (v["qc"], v["sc"])),
                                 (got[5], (v["d"], v["sd"]), (v["a"], v["sa"]))):
        for e in range(E):
            at = v["group"] == e
            if at.any():
                x, y = R.values(p[at], sp[at]), R.values(q[at], sq[at])
                tol = (x.abs().t() @ y.abs()) * (2.0 ** -8 * 1.01 + (len(x) + 4) * 2.0 ** -24)
                ref = x.t() @ y
                assert ((dw[e].double() - ref).abs() <= tol + R.HALF[dw.dtype] * 1.01 * ref.abs()).all()


def test_a_captured_step_with_other_choices():
    """Captured once, replayed with other tokens, weights and experts, eager steps between."""
    m = Layer(150, 512, 256, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = m.step()
    n = m.n
    for i in range(4):
        m.x.copy_(n(150, 512))
        m.go.copy_(n(150, 512))
        m.w13.copy_(n(E, 512, 512) * 512 ** -0.5)
        m.ids.copy_(torch.rand(150, E - i % 3, generator=m.g, device=DEV).argsort(1)[:, :CHOICES] + i % 3)
        want = m.step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)
