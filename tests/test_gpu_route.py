"""The gate on the GPU (dg_moe_route, dg_moe_route_backward, moe_route) against the plain
64-bit form: ids and counts equal, weights, loss and gradients within bounds derived from
the arithmetic; rows with nothing left, ties, infinities and NaN in padding, strides,
streams, graphs; gradients also against central differences of the plain form."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import moe_ref as R  # noqa: E402

DEV = "cuda:0"


def make(T, E, seed, dtype, ld=None, width=1.5, offset=0):
    """Logits on the GPU (rows of ld, the first at `offset` elements of its buffer) and the
    same values on the host."""
    rng = np.random.default_rng(seed)
    ld = ld or E
    buf = torch.full((T * ld + offset + ld,), float("nan"), dtype=dtype, device=DEV)
    z = buf[offset:].as_strided((T, E), (ld, 1))
    host = torch.from_numpy((width * rng.standard_normal((T, E))).astype(np.float32)).to(dtype)
    z.copy_(host)
    return z, host.float().numpy()


def check_forward(z, host, k, *, bias=None, valid=None, score="softmax", normalize=False, scale=1.0,
                  balance=1e-2, **kw):
    print(f"[case] route {tuple(host.shape)} k={k} {z.dtype} {score} normalize={normalize}", flush=True)
    tb = None if bias is None else torch.from_numpy(bias).to(DEV)
    tv = None if valid is None else torch.from_numpy(valid).to(DEV)
    got = dg.dg_moe_route(z, k, bias=tb, row_valid=tv, score=score, normalize=normalize, scale=scale,
                          balance=balance, **kw)
    torch.cuda.synchronize()
    ids, w, counts, loss, coef = (t.cpu().numpy() for t in got)
    r_ids, r_w, r_counts, r_loss, r_coef = R.route(host, k, bias, valid, score, normalize, scale, balance)
    assert np.array_equal(ids, r_ids)
    assert np.array_equal(counts, r_counts)
    tol = R.weight_tolerance(host, host.shape[1])
    assert np.all(np.abs(w - r_w) <= tol * np.abs(r_w) + 1e-36), np.max(np.abs(w - r_w))
    assert np.all(np.abs(coef - r_coef) <= 8 * R.U * np.abs(r_coef))
    # a lane adds the rows of a wave's share, the rest in a tree and over the workgroups
    rows = host.shape[0]
    t_loss = tol + 2 * R.U * (rows / 8192 + 16 + 512 + host.shape[1] / 256 + 16)
    assert abs(float(loss) - r_loss) <= t_loss * abs(r_loss) + 1e-36
    return got


SIZES = [(1, 1, 1), (3, 2, 2), (5, 3, 1), (17, 4, 4), (64, 8, 2), (65, 16, 16), (100, 60, 4), (31, 64, 6),
         (33, 65, 8), (40, 127, 7), (40, 128, 8), (9, 129, 3), (64, 256, 8), (70, 255, 8), (11, 257, 5),
         (12, 512, 16), (7, 513, 2), (5, 1000, 8), (6, 1024, 16), (0, 64, 4)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_forward_sizes(T, E, k, dtype):
    z, host = make(T, E, T + E, dtype)
    rng = np.random.default_rng(E)
    bias = rng.standard_normal(E).astype(np.float32) * np.float32(0.2)
    check_forward(z, host, k)
    check_forward(z, host, k, score="sigmoid", normalize=True, scale=2.5, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_forward_many_rows(score, normalize):
    """More rows than one pass of the grid takes, a third of them padding."""
    T, E = 9001, 24
    z, host = make(T, E, 5, torch.bfloat16)
    valid = (np.random.default_rng(1).random(T) > 0.33).astype(np.uint8)
    z[torch.from_numpy(valid).to(DEV) == 0] = float("nan")
    check_forward(z, host, 3, valid=valid, score=score, normalize=normalize)


def test_forward_grid_strides():
    """Rows of 1024 experts, four rows a workgroup: the workgroups take several blocks."""
    z, host = make(2300, 1024, 6, torch.float32)
    check_forward(z, host, 2, score="softmax")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ld,offset", [(64, 0), (61, 0), (64, 1), (63, 4), (128, 8)])
def test_forward_strides_and_alignment(dtype, ld, offset):
    z, host = make(37, 60, 7, dtype, ld=ld, offset=offset)
    check_forward(z, host, 4)


def test_ties_take_the_lowest_index():
    T, E, k = 40, 200, 8
    host = np.random.default_rng(3).integers(-2, 3, (T, E)).astype(np.float32)
    host[0] = 0.0
    host[1] = -3.5
    host[2, ::2] = -0.0
    host[2, 1::2] = 0.0
    host[3] = 1e-42                         # subnormal
    host[3, 7] = 2e-42
    host[4] = -1e-42
    host[5] = 3.0e38
    host[6] = -3.0e38
    z = torch.from_numpy(host).to(DEV)
    ids = dg.dg_moe_route(z, k, score="sigmoid")[0].cpu().numpy()
    want = np.array([R.choose(r, None, k) for r in host])
    assert np.array_equal(ids, want)
    assert list(ids[0]) == list(range(k)) and list(ids[2]) == list(range(k))
    zb = z.to(torch.bfloat16)
    ids = dg.dg_moe_route(zb, k)[0].cpu().numpy()
    want = np.array([R.choose(r, None, k) for r in zb.float().cpu().numpy()])
    assert np.array_equal(ids, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_keys_of_either_zero_are_equal(dtype):
    """-0 comes out of an addition only where both the logit and the bias are -0."""
    host = np.zeros((3, 40), np.float32)
    host[0] = -0.0
    host[1, ::2] = -0.0
    bias = np.zeros(40, np.float32)
    bias[:20] = -0.0
    bias[30:] = -1.0
    z = torch.from_numpy(host).to(DEV).to(dtype)
    ids = dg.dg_moe_route(z, 8, bias=torch.from_numpy(bias).to(DEV))[0].cpu().numpy()
    assert np.array_equal(ids, np.tile(np.arange(8), (3, 1)))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_closed_experts_and_empty_rows(score):
    T, E, k = 50, 20, 6
    z, host = make(T, E, 8, torch.float32)
    host = host.copy()
    host[0] = -math.inf                    # nothing left
    host[1, 3:] = -math.inf                # fewer than k left
    host[2, :] = -math.inf
    host[2, 19] = -5.0
    host[3] = np.finfo(np.float32).min     # the type's lowest value is a value
    z.copy_(torch.from_numpy(host))
    bias = np.zeros(E, np.float32)
    bias[[4, 9, 13]] = -math.inf           # closed
    for normalize in (False, True):
        check_forward(z, host, k, score=score, normalize=normalize)
        got = check_forward(z, host, k, score=score, normalize=normalize, bias=bias)
        assert not np.isin(got[0].cpu().numpy(), [4, 9, 13]).any()
    bias[:] = -math.inf                    # all closed
    got = check_forward(z, host, k, score=score, bias=bias)
    assert (got[0] == -1).all() and (got[1] == 0).all() and float(got[3]) == 0.0


def test_infinities_and_nan_stay_in_their_rows():
    T, E, k = 12, 40, 4
    z, host = make(T, E, 9, torch.float32)
    host = host.copy()
    host[2, 5] = math.nan
    host[7, 11] = math.inf
    z.copy_(torch.from_numpy(host))
    for score in ("softmax", "sigmoid"):
        ids, w, _, loss, _ = dg.dg_moe_route(z, k, score=score, balance=1.0)
        ids, w = ids.cpu().numpy(), w.cpu().numpy()
        clean = [t for t in range(T) if t not in (2, 7)]
        r_ids, r_w, *_ = R.route(host[clean], k, None, None, score, False, 1.0, 1.0)
        assert np.array_equal(ids[clean], r_ids)
        assert np.all(np.abs(w[clean] - r_w) <= R.weight_tolerance(host, E) * r_w + 1e-36)
        assert 5 not in ids[2] and ids[7, 0] == 11 and (ids >= 0).all() and (ids < E).all()
        assert math.isnan(float(loss))
        if score == "softmax":
            assert np.isnan(w[2]).all() and np.isnan(w[7]).all()
        else:
            assert np.isfinite(w).all() and w[7, 0] == 1.0


def test_all_rows_padding():
    z = torch.full((30, 16), float("nan"), device=DEV)
    valid = torch.zeros(30, dtype=torch.bool, device=DEV)
    ids, w, counts, loss, coef = dg.dg_moe_route(z, 2, row_valid=valid, balance=1.0)
    assert (ids == -1).all() and (w == 0).all() and (counts == 0).all()
    assert float(loss) == 0.0 and (coef == 0).all()
    g = dg.dg_moe_route_backward(z, ids, grad_weights=torch.ones_like(w), coef=coef, row_valid=valid)
    assert (g == 0).all()


def test_outputs_on_request():
    z, host = make(20, 32, 10, torch.float32)
    ids, w, counts, loss, coef = dg.dg_moe_route(z, 4)
    assert counts is None and loss is None and coef is None
    ids2, w2, counts, loss, coef = dg.dg_moe_route(z, 4, count=True)
    assert torch.equal(ids, ids2) and torch.equal(w, w2) and loss is None and coef is None
    assert np.array_equal(counts.cpu().numpy(), np.bincount(ids.cpu().numpy().ravel(), minlength=32))


@pytest.mark.parametrize("T,E", [(5000, 100), (40000, 64), (700, 1000), (20, 16)])
def test_same_bits_again_whatever_the_workspace_holds(T, E):
    z, _ = make(T, E, 11, torch.float32)
    need = dg.dg_moe_route_workspace_bytes(T, E)
    buf = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
    first = dg.dg_moe_route(z, 8, balance=1.0, workspace=buf[:need])
    for fill in (0, 0xFF, 0x7F):
        buf[:need] = fill
        again = dg.dg_moe_route(z, 8, balance=1.0, workspace=buf[:need])
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert (buf[need:] == 0xAB).all()


def test_other_stream_and_graph():
    z, host = make(700, 48, 12, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = dg.dg_moe_route(z, 4, balance=1.0)
    got = dg.dg_moe_route(z, 4, balance=1.0, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    out = [torch.empty_like(t) for t in want]
    gl = torch.ones((), device=DEV)
    gw = torch.rand_like(want[1])
    want_g = dg.dg_moe_route_backward(z, want[0], grad_weights=gw, coef=want[4], grad_loss=gl)
    grad = torch.empty_like(z)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dg.dg_moe_route(z, 4, balance=1.0, ids=out[0], weights=out[1], counts=out[2], loss=out[3],
                        coef=out[4])
        dg.dg_moe_route_backward(z, out[0], grad_weights=gw, coef=out[4], grad_loss=gl, grad_logits=grad)
    for _ in range(4):
        for t in out + [grad]:
            t.zero_()
        dg.dg_moe_route(z, 2, balance=1.0)             # eager work in between
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
        assert torch.equal(want_g, grad)


# ---------------------------------------------------------------------------- backward
def check_backward(T, E, k, dtype, score, normalize, seed, parts="both", ld=None, valid=None, bias=None):
    print(f"[case] backward {T}x{E} k={k} {dtype} {score} normalize={normalize} {parts}", flush=True)
    z, host = make(T, E, seed, dtype, ld=ld)
    rng = np.random.default_rng(seed + 1)
    scale, gl, balance = 1.7, 0.8, 0.3
    tv = None if valid is None else torch.from_numpy(valid).to(DEV)
    tb = None if bias is None else torch.from_numpy(bias).to(DEV)
    how = dict(score=score, normalize=normalize, scale=scale)
    ids, _, _, _, coef = dg.dg_moe_route(z, k, bias=tb, row_valid=tv, balance=balance, **how)
    gw = rng.standard_normal((T, k)).astype(np.float32)
    use_w, use_l = parts in ("both", "weights"), parts in ("both", "loss")
    g = dg.dg_moe_route_backward(z, ids, row_valid=tv, **how,
                                 grad_weights=torch.from_numpy(gw).to(DEV) if use_w else None,
                                 coef=coef if use_l else None,
                                 grad_loss=torch.tensor(gl, device=DEV) if use_l else None)
    assert g.dtype == dtype and g.shape == z.shape
    g = g.float().cpu().numpy()
    r_ids = ids.cpu().numpy()
    r_coef = coef.cpu().numpy().astype(np.float64)
    gl32 = float(np.float32(gl))
    want, size = R.route_grad(host, r_ids, gw if use_w else None, r_coef if use_l else None, gl32, valid,
                              score, normalize, float(np.float32(scale)))
    rel = 3 * R.weight_tolerance(host, E)       # scores, their sums and products of those
    tol = rel * size + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0) + 1e-36
    assert np.all(np.abs(g - want) <= tol), np.max(np.abs(g - want) / tol)
    # the formula against central differences of the plain form
    live = [t for t in range(T) if valid is None or valid[t]]
    for t in live[:3]:
        for e in {0, E // 2, E - 1, max(int(r_ids[t, 0]), 0)}:
            h = 1e-5
            up, dn = host[t].astype(np.float64), host[t].astype(np.float64)
            up[e] += h
            dn[e] -= h
            a = (gw[t].astype(np.float64) * use_w, r_coef * use_l, gl32, score, normalize,
                 float(np.float32(scale)))
            d = (R.route_loss(up, r_ids[t], *a) - R.route_loss(dn, r_ids[t], *a)) / (2 * h)
            # h^2 of the third derivative (a few times the size), and cancellation in 64 bits
            assert abs(d - want[t, e]) <= 1e-9 * (1 + np.abs(gw[t]).sum() * 8)
            assert abs(g[t, e] - d) <= tol[t, e] + 1e-9 * (1 + np.abs(gw[t]).sum() * 8)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 1), (20, 8, 2), (65, 60, 4), (33, 64, 6), (12, 100, 8),
                                   (64, 256, 8), (9, 300, 16), (5, 1024, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_backward_sizes(T, E, k, score, normalize):
    check_backward(T, E, k, torch.float32, score, normalize, T + E)
    check_backward(T, E, k, torch.bfloat16, score, normalize, T + E + 1)


@pytest.mark.parametrize("parts", ["weights", "loss"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_parts(parts, score):
    check_backward(30, 40, 4, torch.float32, score, True, 3, parts=parts)


def test_backward_padding_strides_and_missing_choices():
    valid = (np.arange(50) % 3 != 0).astype(np.uint8)
    bias = np.full(20, -math.inf, np.float32)
    bias[:3] = 0.0                         # fewer open experts than choices
    for score in ("softmax", "sigmoid"):
        check_backward(50, 20, 5, torch.float32, score, True, 4, ld=23, valid=valid, bias=bias)


def test_backward_many_rows():
    check_backward(3000, 1000, 3, torch.float32, "softmax", False, 6)


def test_backward_empty_row_and_wide_gradient():
    z = torch.full((4, 10), -math.inf, device=DEV)
    z[1:] = 0.5
    ids, w, _, _, coef = dg.dg_moe_route(z, 2, normalize=True, balance=1.0)
    wide = torch.full((4, 16), 7.0, device=DEV)
    dg.dg_moe_route_backward(z, ids, grad_weights=torch.ones_like(w), coef=coef, normalize=True,
                             grad_logits=wide[:, 3:13])
    assert (wide[0, 3:13] == 0).all() and torch.isfinite(wide).all()
    assert (wide[:, :3] == 7).all() and (wide[:, 13:] == 7).all()


def test_autograd():
    z, host = make(60, 32, 13, torch.float32)
    z = z.clone().requires_grad_()
    ids, w, counts, loss = dg.moe_route(z, 4, score="sigmoid", normalize=True, scale=2.0, balance=0.5)
    assert not ids.requires_grad and not counts.requires_grad
    gw = torch.rand_like(w)
    ((w * gw).sum() + 3.0 * loss).backward()
    coef = dg.dg_moe_route(z.detach(), 4, score="sigmoid", normalize=True, scale=2.0, balance=0.5)[4]
    want = dg.dg_moe_route_backward(z.detach(), ids, grad_weights=gw, coef=coef,
                                    grad_loss=torch.tensor(3.0, device=DEV), score="sigmoid",
                                    normalize=True, scale=2.0)
    assert torch.equal(z.grad, want)
    z.grad = None
    dg.moe_route(z, 4, balance=0.5)[3].backward()
    assert torch.isfinite(z.grad).all() and z.grad.abs().sum() > 0
    # a second derivative is refused, not left out
    g, = torch.autograd.grad(dg.moe_route(z, 4, balance=0.5)[3], z, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_refusals():
    z = torch.zeros(8, 16, device=DEV)
    with pytest.raises(dg.DGError):
        dg.dg_moe_route(z, 17)
    with pytest.raises(dg.DGError):
        dg.dg_moe_route(z, 0)
    with pytest.raises(dg.DGError):
        dg.dg_moe_route(torch.zeros(2, 1025, device=DEV), 2)
    with pytest.raises(TypeError):
        dg.dg_moe_route(z.half(), 2)
    with pytest.raises(ValueError):
        dg.dg_moe_route(z, 2, score="tanh")
    with pytest.raises(ValueError):
        dg.dg_moe_route(z.t(), 2)
    with pytest.raises(ValueError):
        dg.dg_moe_route(z, 2, bias=torch.zeros(15, device=DEV))
    with pytest.raises(ValueError):
        dg.dg_moe_route(z, 2, loss=torch.zeros((), device=DEV))
    with pytest.raises(ValueError):
        dg.dg_moe_route(z.cpu(), 2)
    with pytest.raises(dg.DGError):
        dg.dg_moe_route(z.repeat(500, 1), 2, count=True,
                        workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        dg.dg_moe_route_backward(z, torch.zeros(8, 2, device=DEV), coef=torch.zeros(16, device=DEV))
