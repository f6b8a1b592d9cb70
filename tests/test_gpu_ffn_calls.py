"""Calls of the feed-forward operators that a program may make and the other tests do not:
workspaces of just the size asked for, gradients as views, tiny scales, a captured training step,
several threads on one stream, launches in slices and offsets past 32 bits."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import ffn_ref as R  # noqa: E402

DEV = "cuda:0"
BF, F = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device=DEV)


def same(a, b):
    return all(p is q is None or torch.equal(p.float(), q.float()) for p, q in zip(a, b))


def guarded(need):
    """A workspace of need bytes that hold NaN, between bytes that no call may touch."""
    whole = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=DEV)
    return whole, whole[256:256 + need]


def untouched(whole):
    return bool((whole[:256] == 0xFF).all() and (whole[-256:] == 0xFF).all())


@pytest.mark.parametrize("kind,rows,N,K,G", [("dense", 1, 2048, 7168, 1), ("dense", 64, 256, 2048, 1),
                                             ("dense", 100, 1152, 1024, 1), ("masked", 33, 384, 1024, 3),
                                             ("masked", 130, 256, 4096, 2)])
def test_gated_workspace(kind, rows, N, K, G):
    n = gen(rows)
    b, sb = R.quantise_weight(n(G, 2 * N, K) * K ** -0.5)
    a, sa = R.quantise(n(G, rows, K))
    need = dg.dg_gated_workspace_bytes(dg.DG_MASKED if kind == "masked" else dg.DG_DENSE, rows, N, K, G)
    whole, ws = guarded(need)
    if kind == "masked":
        counts = torch.tensor([rows, 0, rows // 2][:G], dtype=torch.int32, device=DEV)
        run = lambda **k: dg.dg_grouped_gated_fp8_masked(a, sa, b, sb, counts, **k)  # noqa: E731
    else:
        run = lambda **k: dg.dg_gated_fp8_nt(a[0], sa[0], b[0], sb[0], save=True, **k)  # noqa: E731
    assert same(run(workspace=ws), run()) and untouched(whole)
    if need:                                   # where the sums are split
        with pytest.raises(dg.DGError, match="WORKSPACE"):
            run(workspace=ws[:need - 16])


@pytest.mark.parametrize("T,K", [(1, 128), (517, 2048), (3000, 384)])
def test_norm_backward_workspace(T, K):
    n = gen(T)
    x, dy, w = n(T, K), n(T, K), n(K)
    rstd = dg.dg_rms_norm_fp8(x, w, codes=False, save=True)[4]
    whole, ws = guarded(dg.dg_rms_norm_backward_workspace_bytes(T, K))
    assert same(dg.dg_rms_norm_backward(dy, x, rstd, w, workspace=ws), dg.dg_rms_norm_backward(dy, x, rstd, w))
    assert untouched(whole)


@pytest.mark.parametrize("T,N,K,G", [(5000, 128, 256, 1), (2500, 384, 128, 2)])
def test_wgrad_workspace(T, N, K, G):
    n = gen(T)
    ops = (*R.quantise(n(T, N)), *R.quantise(n(T, K)))
    need = dg.dg_wgrad_workspace_bytes(T, N, K, G)
    assert need > 0
    whole, ws = guarded(need)
    if G == 1:
        run = lambda **k: (dg.dg_wgrad_fp8(*ops, **k),)  # noqa: E731
    else:
        idx = (torch.arange(T, device=DEV) // 1280).int()
        run = lambda **k: (dg.dg_grouped_wgrad_fp8_contiguous(*ops, idx, G, **k),)  # noqa: E731
    assert same(run(workspace=ws), run()) and untouched(whole)


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("dtype", [BF, F])
def test_gradients_as_views(T, dtype):
    """Gradients that reach the block as torch makes them: broadcast (a sum's), turned, with rows
    apart at any distance."""
    n = gen(T)
    K, N, M = 256, 128, 384
    w13, w2 = n(2 * N, K) * K ** -0.5, n(M, N) * N ** -0.5
    x, r = n(T, K).to(dtype).requires_grad_(), n(T, K).to(dtype).requires_grad_()

    def grads(go, gh):
        out, h = dg.gated_ffn(x, w13, w2, residual=r)
        return torch.autograd.grad([out, h], [x, r], [go, gh])

    go, gh = n(T, M).to(BF), n(T, K).to(dtype)
    want = grads(go, gh)
    assert same(grads(go.t().contiguous().t(), gh.t().contiguous().t()), want)
    wide_o, wide_h = torch.zeros(T, M + 3, device=DEV, dtype=BF), torch.zeros(T, K + 5, device=DEV, dtype=dtype)
    wide_o[:, 3:], wide_h[:, 5:] = go, gh
    assert same(grads(wide_o[:, 3:], wide_h[:, 5:]), want)
    ones = grads(torch.ones_like(go), torch.ones_like(gh))
    one = torch.ones((), device=DEV)
    assert same(grads(one.to(BF).expand(T, M), one.to(dtype).expand(T, K)), ones)
    out, h = dg.gated_ffn(x, w13, w2, residual=r)
    assert same(torch.autograd.grad(out.sum() + h.sum(), [x, r]), ones)


@pytest.mark.parametrize("exponent", [-70, -100, -124])
def test_tiny_values(exponent):
    """Blocks whose scales have no reciprocal in fp32, or nearly none."""
    n = gen(3)
    x, w = n(9, 384), 2.0 ** exponent * (1 + 0.1 * n(384))
    q, s, h, _, rstd = dg.dg_rms_norm_fp8(x, w, save=True)
    x64 = x.double()
    y = x64 * (x64.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.double()
    # h rstd w: the sum's 384 roundings (squares have one sign), halved by the root, and those of
    # the mean, the root, the quotient and two products
    err = 256 * 2.0 ** -24 * y.abs()
    R.check_codes(q, s, y, err, "e4m3")
    gu, sgu = R.quantise(n(9, 256))
    dh = 2.0 ** exponent * n(9, 128)
    D, sD = dg.dg_gated_backward(dh, gu, sgu)
    v = R.values(gu, sgu)
    g, u = v[:, :128], v[:, 128:]
    sig = torch.sigmoid(g)
    want = torch.cat((dh.double() * u * (sig + g * sig * (1 - sig)), dh.double() * g * sig), 1)
    # the sigmoid to 2^-18 (its argument's rounding, exp, reciprocal), and a few products
    size = torch.cat((dh.double().abs() * u.abs() * (1 + g.abs()), dh.double().abs() * g.abs()), 1)
    R.check_codes(D, sD, want, size * 2.0 ** -18, "e4m3")


def test_captured_training_step():
    """Forward and backward pass captured together on leaves that have no other graph, and replayed
    on new inputs with eager steps on leaves of their own between the replays."""
    n = gen(11)
    T, K, N, M = 200, 512, 256, 512
    data = [n(T, K).to(BF), n(T, K).to(BF), 1 + 0.1 * n(K), n(2 * N, K) * K ** -0.5, n(M, N) * N ** -0.5]
    go, gh = n(T, M).to(BF), n(T, K).to(BF)

    def step(values):
        x, r, w, w13, w2 = leaves = [v.detach().requires_grad_() for v in values]
        out, h = dg.gated_ffn(x, w13, w2, residual=r, norm_weight=w)
        return [out.detach(), h.detach(), *torch.autograd.grad([out, h], leaves, [go, gh])]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(data)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(data)
    for i in range(4):
        data[0].copy_(n(T, K))
        data[3].copy_(n(2 * N, K) * K ** -0.5)
        go.copy_(n(T, M))
        want = step(data)
        graph.replay()
        torch.cuda.synchronize()
        assert same(held, want)


def test_threads_on_one_stream():
    """Calls of several threads on one stream, which share its kept workspaces."""
    n = gen(5)
    jobs = []
    for M in (1, 40, 100):
        a, sa = R.quantise(n(M, 4096))
        b, sb = R.quantise_weight(n(512, 4096) / 64)
        p = (*R.quantise(n(3000 + M, 128)), *R.quantise(n(3000 + M, 256)))
        x, w = n(600, 1024), n(1024)
        rstd = dg.dg_rms_norm_fp8(x, w, codes=False, save=True)[4]

        def run(a=a, sa=sa, b=b, sb=sb, p=p, x=x, rstd=rstd, w=w):
            return (*dg.dg_gated_fp8_nt(a, sa, b, sb, save=True), dg.dg_wgrad_fp8(*p),
                    *dg.dg_rms_norm_backward(x, x, rstd, w))

        jobs.append((run, run()))
    torch.cuda.synchronize()
    bad = []

    def work(run, want):
        for _ in range(20):
            if not same(run(), want):
                bad.append(1)

    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad


def test_norm_rows_past_a_launch_and_32_bits():
    """More rows than one launch takes, whose offsets in elements pass 32 bits."""
    T, K, wide = (1 << 20) + 5, 128, 4096
    n = gen(1)
    x = torch.empty(T, wide, device=DEV, dtype=BF)[:, :K]
    x.copy_(n(T, K))
    r = n(T, K).to(BF)
    w = 1 + 0.1 * n(K)
    whole = dg.dg_rms_norm_fp8(x, w, residual=r, H=x, bf16=True, save=True)
    for at in (slice(0, 40), slice((1 << 20) - 20, T)):
        # H took X's place: its rows again, without a residual
        part = dg.dg_rms_norm_fp8(x[at], w, bf16=True, save=True)
        assert same([v[at] for v in whole], part)
    gx, gw = dg.dg_rms_norm_backward(r, x, whole[4], w, grad_x=x)
    at = slice(T - 40, T)
    h = whole[3][at]
    assert gx[at].shape == h.shape and gx[at].isfinite().all() and gw.isfinite().all()


def wgrad_check(got, p, sp, q, sq, before=None):
    """A gradient against the sum in 64 bits."""
    p, q = R.values(p, sp), R.values(q, sq)
    want, mag = p.t() @ q, p.abs().t() @ q.abs()
    if before is not None:
        want, mag = want + before.double(), mag + before.double().abs()
    # one factor of each product is rounded to bf16 (2^-8, its scales' product before), the sum of
    # the products to fp32 at each step, the result to its type
    tol = mag * (2.0 ** -8 * 1.01 + (p.shape[0] + 4) * 2.0 ** -24) + R.HALF[got.dtype] * want.abs() * 1.01
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [1, 63, 65, 130, 333, 1000])
def test_wgrad_large_tiles(T, dtype):
    """Tiles of 256 x 256 that the last columns of both matrices leave half empty."""
    N, K = 4224, 2432
    fp, fq = [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")][T % 4]
    n = gen(T)
    ops = (*R.quantise(0.01 * n(T, N) * torch.exp(n(T, 1)), fp), *R.quantise(n(T, K), fq))
    wgrad_check(dg.dg_wgrad_fp8(*ops, dtype=dtype), *ops)
    old = 0.01 * n(N, K).to(dtype)
    wgrad_check(dg.dg_wgrad_fp8(*ops, old.clone(), accumulate=True), *ops, before=old)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("order,tail", [([0, 1], 0), ([1, 0, 1], 61), ([1], 7)])
def test_wgrad_large_tiles_of_groups(order, tail, dtype):
    """The same of groups: one's rows in two places, one without rows, NaN in rows that count
    nowhere, a last block that ends early."""
    N, K, G = 2304, 2176, 2
    n = gen(tail)
    idx = []
    for i, g in enumerate(order):
        rows = [200, 1, 77][i]
        blocks = -(-rows // 128) * 128
        idx += [g] * rows + [-1] * (blocks - rows)
    idx += [0] * tail
    idx = torch.tensor(idx, dtype=torch.int32, device=DEV)
    T = idx.numel()
    p, sp = R.quantise(0.01 * n(T, N) * torch.exp(n(T, 1)))
    q, sq = R.quantise(n(T, K))
    p.view(torch.uint8)[idx < 0] = 0x7F
    sq[idx < 0] = float("nan")
    got = dg.dg_grouped_wgrad_fp8_contiguous(p, sp, q, sq, idx, G, dtype=dtype)
    for g in range(G):
        at = (idx == g).nonzero()[:, 0]
        if at.numel():
            wgrad_check(got[g], p[at], sp[at], q[at], sq[at])
        else:
            assert (got[g] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [1, 127, 128, 129, 513, 1024, 1025])
@pytest.mark.parametrize("K", [128, 2048, 2176, 4224, 8192, 8320])
def test_norm_backward_sizes(T, K, dtype):
    """Rows and widths on both sides of what the backward pass goes by, with rows apart, and in the
    gradient's own place."""
    n = gen(T + K)
    h = torch.zeros(T, K + 8, device=DEV, dtype=dtype)[:, :K]
    h.copy_(n(T, K))
    dy, gh, w = n(T, K).to(dtype), n(T, K).to(dtype), 1 + 0.1 * n(K)
    rstd = dg.dg_rms_norm_fp8(h, w, codes=False, save=True)[4]
    dx, dw = dg.dg_rms_norm_backward(dy, h, rstd, w, grad_h=gh)
    H, Y, r = h.double(), dy.double(), rstd.double()[:, None]
    g = Y * w.double()
    m = (g * H).sum(1, keepdim=True) / K
    want, mean_size = r * (g - H * r * r * m) + gh.double(), (g * H).abs().sum(1, keepdim=True) / K
    size = r * (g.abs() + H.abs() * r * r * mean_size) + gh.double().abs()
    # the mean's sum of K products has K roundings at most, the rest a few; the result its type's
    assert ((dx.double() - want).abs() <= (K + 16) * 2.0 ** -24 * size + R.HALF[dtype] * 1.01 * want.abs()).all()
    terms = Y * H * r
    assert ((dw.double() - terms.sum(0)).abs() <= (T + 4) * 2.0 ** -24 * terms.abs().sum(0)).all()
    own = dy.clone()
    assert same(dg.dg_rms_norm_backward(own, h, rstd, w, grad_h=gh, grad_x=own), (dx, dw))
    assert same(dg.dg_rms_norm_backward(dy, h, rstd, w, grad_h=gh, grad_weight=False), (dx, None))


# (rows, group) runs; a group's segment starts on a multiple of 128 where the call is to write it
RUNS = {"one": [(77, 1)], "two": [(128, 0), (100, 2)], "holes": [(5, -1), (123, 0), (130, 2), (126, -1), (128, 7), (60, 0)],
        "again": [(40, 2), (88, 0), (256, 1), (129, 2)], "none": [(300, -1)],
        "many": [(256, 0), (200, 1), (56, -1), (384, 2), (128, 1), (300, 0), (20, 3)]}


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("K", [1024, 4096])
@pytest.mark.parametrize("runs", list(RUNS))
def test_gated_contiguous_few_tiles(runs, K, save):
    """The contiguous form where its tiles are split: blocks whose first row names no group, rows that
    do not follow their block's, the same group in several places, out-of-range groups, NaN in
    every row that is not written."""
    from tests.test_gpu_gated import check
    N, G = 256, 3
    n = gen(K + len(runs))
    idx = torch.cat([torch.full((r,), g, dtype=torch.int32) for r, g in RUNS[runs]]).to(DEV)
    T = idx.numel()
    assert dg.dg_gated_workspace_bytes(dg.DG_CONTIGUOUS, T, N, K, G) > 0 or K < 4096
    lead = idx[torch.arange(T, device=DEV) // 128 * 128]
    written = (idx == lead) & (idx >= 0) & (idx < G)
    a, sa = R.quantise(n(T, K))
    b, sb = R.quantise_weight(n(G, 2 * N, K) * K ** -0.5)
    a.view(torch.uint8)[~written] = 0x7F
    sa[~written] = float("nan")
    H, GU = (torch.full((T, m), 0x33, dtype=torch.uint8, device=DEV) for m in (N, 2 * N))
    sH, sGU = torch.full((T, N // 128), -5.0, device=DEV), torch.full((T, N // 64), -5.0, device=DEV)
    kept = dict(GU=GU, sGU=sGU) if save else {}
    out = dg.dg_grouped_gated_fp8_contiguous(a, sa, b, sb, idx, H, sH, activation="gelu", **kept)
    for t, v in ((H, 0x33), (sH, -5)) + (((GU, 0x33), (sGU, -5)) if save else ()):
        assert (t[~written] == v).all()
    for g in range(G):
        at = (written & (idx == g)).nonzero()[:, 0]
        if at.numel():
            check(*(o if o is None else o[at] for o in out), R.values(a[at], sa[at]), R.weight_values(b[g], sb[g]),
                  "gelu", "e4m3", f"group {g}")
    whole, ws = guarded(dg.dg_gated_workspace_bytes(dg.DG_CONTIGUOUS, T, N, K, G))
    again = dg.dg_grouped_gated_fp8_contiguous(a, sa, b, sb, idx, H.clone(), sH.clone(), activation="gelu", save=save,
                                               workspace=ws)
    assert untouched(whole) and torch.equal(again[0][written].float(), out[0][written].float())
    assert torch.equal(again[1][written], out[1][written])


def test_split_calls_in_a_graph_with_new_rows():
    """Decode calls whose tiles are split, captured once and replayed with other counts and group
    indices, all and none of the rows among them, with eager calls between."""
    n = gen(21)
    G, cap, T, N, K = 4, 150, 400, 256, 4096
    b, sb = R.quantise_weight(n(G, 2 * N, K) * K ** -0.5)
    am, sam = R.quantise(n(G, cap, K))
    ac, sac = R.quantise(n(T, K))
    counts = torch.tensor([3, 0, 150, 70], dtype=torch.int32, device=DEV)
    idx = torch.tensor([0] * 128 + [2] * 200 + [-1] * 72, dtype=torch.int32, device=DEV)
    assert dg.dg_gated_workspace_bytes(dg.DG_MASKED, cap, N, K, G) > 0
    assert dg.dg_gated_workspace_bytes(dg.DG_CONTIGUOUS, T, N, K, G) > 0

    def step():
        m = dg.dg_grouped_gated_fp8_masked(am, sam, b, sb, counts)
        c = dg.dg_grouped_gated_fp8_contiguous(ac, sac, b, sb, idx, save=True)
        return [t.view(torch.uint8) if t.element_size() == 1 else t for t in (*m[:2], *c)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for c, i in (([150] * 4, [1] * 400), ([0] * 4, [-1] * 400), ([1, 2, 129, 0], [3] * 128 + [3] * 272),
                 ([-7, 500, 64, 65], [0] * 100 + [-1] * 28 + [9] * 128 + [2] * 144)):
        counts.copy_(torch.tensor(c, dtype=torch.int32))
        idx.copy_(torch.tensor(i, dtype=torch.int32))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(held, want):
            assert torch.equal(p, q)
