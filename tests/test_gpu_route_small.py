"""The gate where the scores that count are tiny: normalized weights are quotients of scores, and
they and their gradients keep their precision where the scores themselves leave fp32 (choices
far below closed experts under softmax, low logits under sigmoid); so do the sigmoid's shares in
the balance loss."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import moe_ref as R  # noqa: E402
from tests.test_gpu_route import DEV, check_forward  # noqa: E402


def case(score, E, low, seed):
    """Logits of 24 rows and a bias.  softmax: the first half of the experts has logits around 0
    and is closed, the others lie around `low`; sigmoid: all around `low`, but for two rows
    around 0, two with one open expert around 0 among the low ones."""
    rng = np.random.default_rng(seed)
    z = (2.0 * rng.standard_normal((24, E))).astype(np.float32)
    bias = np.zeros(E, np.float32)
    if score == "softmax":
        z[:, E // 2:] += low
        z[0, E // 2] = 0.5                                 # an open one beside the closed
        bias[: E // 2] = -math.inf
    else:
        z[2:] += low
        z[2, 1] = z[3, E - 1] = 0.25
        bias[:] = 0.1 * rng.standard_normal(E)
    return z, bias


CASES = [("softmax", 256, -70), ("softmax", 256, -85), ("softmax", 64, -88), ("softmax", 60, -120),
         ("softmax", 1000, -300), ("sigmoid", 256, -20), ("sigmoid", 64, -80), ("sigmoid", 9, -85),
         ("sigmoid", 60, -100), ("sigmoid", 256, -300), ("sigmoid", 1024, -550)]


def on_gpu(z, dtype):
    t = torch.from_numpy(z).to(DEV).to(dtype)
    return t, t.float().cpu().numpy()


@pytest.mark.parametrize("score,E,low", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k,scale", [(1, 1.0), (4, 2.5), (8, 1000.0)])
def test_normalized_weights_and_loss(score, E, low, dtype, k, scale):
    if k > E // 2:
        pytest.skip("more choices than open experts")
    z, bias = case(score, E, low, E + k)
    t, host = on_gpu(z, dtype)
    ids, w, *_ = check_forward(t, host, k, bias=bias, score=score, normalize=True, scale=scale)
    # each row's weights are a partition of the scale
    tol = R.weight_tolerance(host, E)
    assert np.all(np.abs(w.double().sum(1).cpu().numpy() - scale) <= tol * scale)
    if score == "sigmoid":
        check_forward(t, host, k, score=score, normalize=True, scale=scale)


@pytest.mark.parametrize("score,E,low", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k,scale", [(1, 1.0), (4, 2.5), (8, 1000.0)])
def test_gradients(score, E, low, dtype, k, scale):
    if k > E // 2:
        pytest.skip("more choices than open experts")
    z, bias = case(score, E, low, E + k)
    t, host = on_gpu(z, dtype)
    how = dict(score=score, normalize=True, scale=scale)
    ids, _, _, _, coef = dg.dg_moe_route(t, k, bias=torch.from_numpy(bias).to(DEV), balance=0.3, **how)
    gw = np.random.default_rng(k).standard_normal((24, k)).astype(np.float32)
    g = dg.dg_moe_route_backward(t, ids, grad_weights=torch.from_numpy(gw).to(DEV), coef=coef, **how)
    g = g.float().cpu().numpy()
    r_ids, r_coef = ids.cpu().numpy(), coef.cpu().numpy().astype(np.float64)
    s32 = float(np.float32(scale))
    want, size = R.route_grad(host, r_ids, gw, r_coef, 1.0, None, score, True, s32)
    tol = 3 * R.weight_tolerance(host, E) * size + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0) \
        + 1e-36
    assert np.all(np.abs(g - want) <= tol), np.max(np.abs(g - want) / tol)
    # central differences of the plain form: h^2 of the third derivative, cancellation in 64 bits
    for row in (0, 2, 23):
        for e in {int(r_ids[row, 0]), int(r_ids[row, k - 1]), 0}:
            h = 1e-5
            up, dn = host[row].astype(np.float64), host[row].astype(np.float64)
            up[e] += h
            dn[e] -= h
            a = (gw[row].astype(np.float64), r_coef, 1.0, score, True, s32)
            d = (R.route_loss(up, r_ids[row], *a) - R.route_loss(dn, r_ids[row], *a)) / (2 * h)
            assert abs(g[row, e] - d) <= tol[row, e] + 1e-9 * s32 * (1 + np.abs(gw[row]).sum() * 8)


def test_a_nan_makes_normalized_softmax_weights_nan():
    """The scores of its row are NaN, and so are their quotients, chosen or not."""
    z = torch.randn(6, 40, device=DEV)
    z[1, 7] = math.nan
    z[4, 3] = math.inf
    ids, w, *_ = dg.dg_moe_route(z, 4, normalize=True)
    assert 7 not in ids[1].tolist()
    nan = torch.tensor([False, True, False, False, True, False], device=DEV)
    assert torch.isnan(w[nan]).all() and torch.isfinite(w[~nan]).all()


@pytest.mark.parametrize("E,low", [c[1:] for c in CASES if c[0] == "sigmoid"])
@pytest.mark.parametrize("parts", ["both", "loss"])
def test_sigmoid_shares_in_the_loss(E, low, parts):
    """Weights that are the scores themselves, or no gradient of theirs: the loss's part alone keeps
    its precision, and the weights' is what the scores are."""
    z, bias = case("sigmoid", E, low, E)
    t, host = on_gpu(z, torch.float32)
    ids, _, _, _, coef = check_forward(t, host, 4, bias=bias, score="sigmoid", balance=0.3)
    gw = np.random.default_rng(E).standard_normal((24, 4)).astype(np.float32) if parts == "both" else None
    g = dg.dg_moe_route_backward(t, ids, grad_weights=None if gw is None else torch.from_numpy(gw).to(DEV),
                                 coef=coef, score="sigmoid")
    want, size = R.route_grad(host, ids.cpu().numpy(), gw, coef.cpu().numpy().astype(np.float64), 1.0, None,
                              "sigmoid", False, 1.0)
    tol = 3 * R.weight_tolerance(host, E) * size + 1e-36
    assert np.all(np.abs(g.cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("score,E,low", [c for c in CASES if c[1] <= 256])
def test_rows_beside_tiny_ones_keep_their_bits(score, E, low):
    """Ordinary rows of a wave are not touched by what its tiny rows take."""
    z, bias = case(score, E, low, E)
    rng = np.random.default_rng(5)
    plain = rng.standard_normal(z.shape).astype(np.float32)
    how = dict(score=score, normalize=True)
    gw = torch.from_numpy(rng.standard_normal((48, 4)).astype(np.float32)).to(DEV)

    def rows(z, gw):
        t = torch.from_numpy(z).to(DEV)
        ids, w, *_ = dg.dg_moe_route(t, 4, bias=torch.from_numpy(bias).to(DEV), **how)
        coef = torch.linspace(0.0, 0.1, E, device=DEV)
        return ids, w, dg.dg_moe_route_backward(t, ids, grad_weights=gw, coef=coef, **how)

    mixed = np.empty((48, E), np.float32)
    mixed[0::2], mixed[1::2] = plain, z
    for got, alone in zip(rows(mixed, gw), rows(plain, gw[0::2].contiguous())):
        assert torch.equal(got[0::2], alone)
    for got, alone in zip(rows(mixed, gw), rows(z, gw[1::2].contiguous())):
        assert torch.equal(got[1::2], alone)


@pytest.mark.parametrize("normalize", [False, True])
def test_a_nan_stays_its_own_in_a_sigmoid_row_without_the_loss(normalize):
    """Weights under sigmoid come from their own logits, and so do their gradients; the loss's
    shares, and with them its gradient, meet the whole row."""
    z = torch.randn(9, 40, device=DEV)
    z[3, 7] = -math.inf                     # a score of 0, in no choice
    ids, w, _, _, coef = dg.dg_moe_route(z, 4, score="sigmoid", normalize=normalize, balance=1.0)
    gw = torch.randn(9, 4, device=DEV)
    how = dict(score="sigmoid", normalize=normalize)
    want = dg.dg_moe_route_backward(z, ids, grad_weights=gw, **how)
    assert torch.isfinite(want).all()
    z[3, 7] = math.nan
    again = dg.dg_moe_route(z, 4, **how)
    assert torch.equal(again[0], ids) and torch.equal(again[1], w)
    got = dg.dg_moe_route_backward(z, ids, grad_weights=gw, **how)
    others = torch.ones_like(z, dtype=torch.bool)
    others[3, 7] = False
    assert torch.equal(got[others], want[others])
    got = dg.dg_moe_route_backward(z, ids, grad_weights=gw, coef=coef, **how)
    assert torch.isnan(got[3]).all() and torch.isfinite(got[:3]).all() and torch.isfinite(got[4:]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,ld,at", [(50, 20, 5, 31, 3), (9001, 24, 4, 24, 0), (2300, 1000, 6, 1003, 2),
                                         (700, 8, 3, 9, 1)])
def test_tiny_rows_among_others(score, dtype, T, E, k, ld, at):
    """Every third row tiny, rows inside wider ones, padding, fewer open experts than choices, and
    more rows than the grid takes at once; the gradient too goes into wider rows."""
    rng = np.random.default_rng(T)
    z = rng.standard_normal((T, E)).astype(np.float32)
    bias = np.zeros(E, np.float32)
    closed = rng.permutation(E)[: E - (k - 1)]            # k - 1 are open
    bias[closed] = -math.inf
    z[::3, np.setdiff1d(np.arange(E), closed)] -= 92.0
    if score == "sigmoid":
        z[::3] = z[::3].clip(max=-88.0)
    valid = (rng.random(T) > 0.2).astype(np.uint8)
    wide = torch.full((T, ld), float("nan"), dtype=dtype, device=DEV)
    t = wide[:, at:at + E]
    host = torch.from_numpy(z).to(dtype)
    t.copy_(host)
    t[torch.from_numpy(valid).to(DEV) == 0] = float("nan")
    host = host.float().numpy()
    ids, w, _, _, coef = check_forward(t, host, k, bias=bias, valid=valid, score=score, normalize=True,
                                       scale=2.0)
    assert (ids[:, k - 1] == -1).all()
    gw = rng.standard_normal((T, k)).astype(np.float32)
    out = torch.full((T, ld), 7.0, dtype=dtype, device=DEV)
    dg.dg_moe_route_backward(t, ids, grad_weights=torch.from_numpy(gw).to(DEV), coef=coef, score=score,
                             normalize=True, scale=2.0, row_valid=torch.from_numpy(valid).to(DEV),
                             grad_logits=out[:, at:at + E])
    some = np.unique(np.concatenate([np.arange(min(T, 60)), np.arange(T - 40, T)]))
    want, size = R.route_grad(host[some], ids.cpu().numpy()[some], gw[some],
                              coef.cpu().numpy().astype(np.float64), 1.0, valid[some], score, True, 2.0)
    got = out[:, at:at + E].float().cpu().numpy()
    tol = 3 * R.weight_tolerance(host, E) * size + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0) \
        + 1e-36
    assert np.all(np.abs(got[some] - want) <= tol)
    assert np.isfinite(got).all() and (got[valid == 0] == 0).all()
    rest = torch.ones(ld, dtype=torch.bool, device=DEV)
    rest[at:at + E] = False
    assert (out[:, rest] == 7).all()
