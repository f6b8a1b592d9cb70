"""How the calls of the gate and the adapters take their arguments on the GPU: views that they
refuse, threads that share a stream."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16


def test_a_row_alone_with_strided_columns_is_refused():
    """A single token's logits, x, base, out and gradient, as for more rows."""
    wide = torch.randn(4, 256, device=DEV)
    z = wide[:1, ::2]
    ids = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    coef = torch.zeros(128, device=DEV)
    with pytest.raises(ValueError, match="dense rows"):
        dg.dg_moe_route(z, 2)
    with pytest.raises(ValueError, match="dense rows"):
        dg.dg_moe_route_backward(z, ids, coef=coef)
    with pytest.raises(ValueError, match="dense rows"):
        dg.dg_moe_route_backward(z.contiguous(), ids, coef=coef, grad_logits=wide[1:2, ::2])
    xw = torch.randn(4, 256, device=DEV).to(BF)
    x, strided = xw[:1, :128], xw[:1, ::2]
    A, B = torch.randn(2, 8, 128, device=DEV).to(BF), torch.randn(2, 128, 8, device=DEV).to(BF)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    before = xw.clone()
    for args in ((strided, A, B, one), (x, A, B, one, strided), (x, A, B, one, None, strided)):
        with pytest.raises(ValueError, match="dense rows"):
            dg.dg_lora_bf16(*args)
    assert torch.equal(xw, before)
    # a row of a wider matrix is dense, whatever its row stride
    got = dg.dg_lora_bf16(x, A, B, one)
    assert torch.equal(got, dg.dg_lora_bf16(x.contiguous(), A, B, one))
    assert torch.equal(dg.dg_moe_route(wide[:1, :128], 2)[0], dg.dg_moe_route(wide[:1, :128].contiguous(), 2)[0])


def test_threads_on_one_stream():
    """Threads share the default stream and with it the kept workspace: each call's result is the
    one it has alone, and of a call of several launches none is between another's."""
    rng = torch.Generator(device=DEV)
    rng.manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=rng, device=DEV)

    jobs = []
    for i in range(4):
        z = normal(3000, 64) * (i + 1)
        T = (5, 40, 200, 700)[i]
        x, A, B = normal(T, 512).to(BF), normal(3, 16, 512).to(BF), normal(3, 264, 16).to(BF)
        ids = (torch.arange(T, device=DEV) % 3).int()
        jobs.append((lambda z=z: dg.dg_moe_route(z, 4, balance=1.0),
                     lambda a=(x, A, B, ids): (dg.dg_lora_bf16(*a),)))
    want = [[f() for f in job] for job in jobs]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(jobs))

    def work(i):
        start.wait()
        got = [[f() for f in jobs[i]] for _ in range(30)]
        torch.cuda.synchronize()
        for n, pair in enumerate(got):
            for w, g in zip(want[i], pair):
                if not all(torch.equal(a, b) for a, b in zip(w, g)):
                    wrong.append((i, n))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


@pytest.mark.parametrize("T,E", [(64, 256), (40, 128), (200, 40), (64, 257), (65, 256), (300, 256), (129, 8)])
@pytest.mark.parametrize("k", [1, 3, 8, 16])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_asking_for_counts_changes_no_bits(T, E, k, dtype, score):
    """Calls with counts may take another shape (sigmoid: one workgroup and one launch, at and just
    past the sizes where they do); choices and weights stay what they are."""
    if k > E:
        pytest.skip("more choices than experts")
    g = torch.Generator(device=DEV)
    g.manual_seed(T + E + k)
    z = (2 * torch.randn(T, E, generator=g, device=DEV)).to(dtype)
    z[T // 2] -= 95.0                          # tiny scores
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    for normalize in (False, True):
        for b in (None, bias):
            how = dict(score=score, normalize=normalize, scale=2.5, bias=b)
            ids, w, *_ = dg.dg_moe_route(z, k, **how)
            ids2, w2, counts, *_ = dg.dg_moe_route(z, k, count=True, **how)
            assert torch.equal(ids, ids2) and torch.equal(w, w2)
            assert torch.equal(counts.long(), torch.bincount(ids[ids >= 0].long(), minlength=E))
