"""Low-rank adapters on the GPU (dg_lora_bf16) against the plain 64-bit form: batch sizes
around the 16-row tile, odd widths, every mix of adapters and ranks, rows without one,
other adapters' infinities, strides, in-place bases, offsets past 32 bits, streams, graphs;
and behind the FP8 projection that it stands beside."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402
from tests import moe_ref as R  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16


def bf(rng, *shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(BF)


def host(t):
    return None if t is None else t.float().cpu().numpy()


def strided(t, ld, offset=0, fill=float("nan")):
    """The same matrix on the GPU with rows `ld` apart, starting at element `offset`."""
    buf = torch.full((t.shape[0] * ld + offset + ld,), fill, dtype=t.dtype, device=DEV)
    v = buf[offset:].as_strided(tuple(t.shape), (ld, 1))
    v.copy_(t)
    return v


def make(T, N, K, rank, L, seed):
    rng = np.random.default_rng(seed)
    return dict(x=bf(rng, T, K), A=bf(rng, L, rank, K, scale=K ** -0.5), B=bf(rng, L, N, rank, scale=0.3),
                base=bf(rng, T, N), scales=torch.from_numpy(rng.uniform(0.5, 2, L).astype(np.float32)))


def check(p, ids, ranks=None, scales=True, base=True, what="", **kw):
    T, K = p["x"].shape
    L, rank, _ = p["A"].shape
    N = p["B"].shape[1]
    print(f"[case] lora T={T} N={N} K={K} R={rank} L={L} {what}", flush=True)
    ids = np.asarray(ids, np.int32)
    s = p["scales"] if scales else None
    b = p["base"] if base else None
    t_ranks = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device=DEV)
    got = dg.dg_lora_bf16(p["x"].to(DEV), p["A"].to(DEV), p["B"].to(DEV), torch.from_numpy(ids).to(DEV),
                          None if b is None else b.to(DEV), scales=None if s is None else s.to(DEV),
                          ranks=t_ranks, **kw)
    torch.cuda.synchronize()
    ref, size = R.lora(host(p["x"]), host(p["A"]), host(p["B"]), ids, host(s), ranks, host(b))
    g = host(got).astype(np.float64)
    tol = R.lora_tolerance(ref, size, K)
    assert np.all(np.abs(g - ref) <= tol), np.max(np.abs(g - ref) / tol)
    none = (ids < 0) | (ids >= L)
    if b is not None:
        assert np.array_equal(host(got)[none], host(b)[none])
    else:
        assert (host(got)[none] == 0).all()
    return got


def ids_of(T, L, kind, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full(T, L - 1)
    if kind == "distinct":
        return np.arange(T) % L
    if kind == "segments":
        return np.sort(rng.integers(0, L, T))
    if kind == "mixed":
        return rng.integers(-1, L, T)
    return np.full(T, -1)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 100])
@pytest.mark.parametrize("kind", ["one", "distinct", "mixed", "none"])
def test_batches(T, kind):
    check(make(T, 200, 384, 16, 20, T), ids_of(T, 20, kind, T), what=kind)


@pytest.mark.parametrize("N", [1, 3, 7, 8, 9, 31, 64, 65, 250, 256, 257, 2111])
def test_widths(N):
    check(make(19, N, 256, 16, 5, N), ids_of(19, 5, "mixed"))


@pytest.mark.parametrize("K", [128, 256, 1152, 4096, 4224, 7168, 16384])
def test_depths(K):
    check(make(20, 72, K, 16, 3, K), ids_of(20, 3, "mixed"))
    check(make(1, 72, K, 8, 3, K), [1])


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
def test_ranks_of_storage(rank):
    check(make(40, 136, 512, rank, 6, rank), ids_of(40, 6, "mixed"))


@pytest.mark.parametrize("rank", [8, 16, 40, 64])
def test_ranks_of_adapters(rank):
    """Each adapter its own rank; what A and B hold past it must not count."""
    ranks = [0, 1, 7, 8, 9, rank, rank + 5, -3, rank - 1]
    p = make(50, 90, 256, rank, len(ranks), rank)
    for i, r in enumerate(ranks):
        r = min(max(r, 0), rank)
        p["A"][i, r:] = float("nan")
        p["B"][i, :, r:] = float("inf")
    check(p, ids_of(50, len(ranks), "mixed"), ranks=ranks)


@pytest.mark.parametrize("T,L", [(300, 3), (1093, 24), (1000, 1)])
def test_long_batches(T, L):
    p = make(T, 264, 256, 16, L, T)
    check(p, ids_of(T, L, "segments"), what="segments")
    check(p, ids_of(T, L, "mixed"), what="mixed")


def test_many_rows_of_rank_64():
    check(make(2100, 520, 128, 64, 4, 3), ids_of(2100, 4, "segments"))


@pytest.mark.parametrize("T,K,rank,L", [(2000, 4096, 64, 9), (1500, 2048, 128, 5), (700, 8192, 16, 40),
                                        (4100, 1024, 32, 70), (130, 128, 8, 3), (3000, 1152, 72, 300)])
def test_parts_of_long_batches(T, K, rank, L):
    """Prompts whose ends fall inside tiles, then single rows: items cut into parts of K, even
    and uneven ones."""
    p = make(T, 40, K, rank, L, T + K)
    rng = np.random.default_rng(T)
    prompts = np.sort(rng.integers(0, max(L // 3, 1), T - min(L, T // 4)))
    ids = np.concatenate([prompts, np.arange(min(L, T // 4))])
    check(p, ids, what="prompts and single rows")
    ids[rng.random(T) < 0.8] = -1                # few items
    check(p, ids, what="mostly without an adapter")


def test_one_row_with_an_adapter_among_many():
    p = make(1000, 24, 1024, 16, 3, 21)
    ids = np.full(1000, -1)
    ids[777] = 2
    check(p, ids)


def test_more_rows_than_a_launch_takes():
    T, K, N, rank, L = (1 << 20) + 77, 128, 8, 8, 3
    p = make(1, N, K, rank, L, 22)
    x = torch.randn(T, K, device=DEV, dtype=torch.float32).to(BF)
    base = torch.randn(T, N, device=DEV, dtype=torch.float32).to(BF)
    ids = ((torch.arange(T, device=DEV) // 1000) % (L + 1) - 1).int()
    got = dg.dg_lora_bf16(x, p["A"].to(DEV), p["B"].to(DEV), ids, base)
    torch.cuda.synchronize()
    rows = np.concatenate([np.arange(300), np.arange((1 << 20) - 200, T)])
    ref, size = R.lora(host(x[rows]), host(p["A"]), host(p["B"]), ids.cpu().numpy()[rows], None, None,
                       host(base[rows]))
    assert np.all(np.abs(host(got[rows]) - ref) <= R.lora_tolerance(ref, size, K))
    none = ids < 0
    assert torch.equal(got[none], base[none])


@pytest.mark.parametrize("N", [12544, 12301])
def test_outputs_larger_than_the_caches(N):
    """Outputs of 100 MB and more are stored past the caches, aligned or not."""
    T, K, rank, L = 4200, 128, 8, 3
    p = make(1, N, K, rank, L, 23)
    x = torch.randn(T, K, device=DEV, dtype=torch.float32).to(BF)
    base = torch.randn(T, N, device=DEV, dtype=torch.float32).to(BF)
    ids = ((torch.arange(T, device=DEV) // 700) % (L + 1) - 1).int()
    A, B = p["A"].to(DEV), p["B"].to(DEV)
    got = dg.dg_lora_bf16(x, A, B, ids, base)
    some = torch.arange(1401, device=DEV) * 3                 # the same rows in a smaller call
    some = some[some < T]
    assert (got[ids < 0] == base[ids < 0]).all()
    rows = np.concatenate([np.arange(690, 730), np.arange(T - 40, T)])
    ref, size = R.lora(host(x[rows]), host(p["A"]), host(p["B"]), ids.cpu().numpy()[rows], None, None,
                       host(base[rows]))
    assert np.all(np.abs(host(got[rows]) - ref) <= R.lora_tolerance(ref, size, K))
    less = dg.dg_lora_bf16(x[some], A, B, ids[some], base[some])
    assert (got[some].float() - less.float()).abs().max() <= 2.0 ** -7 * got[some].float().abs().max()


def test_no_scales_no_base():
    p = make(30, 100, 256, 16, 4, 5)
    check(p, ids_of(30, 4, "mixed"), scales=False)
    check(p, ids_of(30, 4, "mixed"), base=False)
    check(p, ids_of(30, 4, "mixed"), base=False, scales=False)


def test_ids_outside_the_adapters():
    p = make(40, 64, 128, 16, 4, 6)
    check(p, [-1, 4, 5, -7, 2 ** 31 - 1, -2 ** 31, 0, 3] * 5)


def test_other_adapters_values_do_not_matter():
    """A row's bits stay what they are whatever the other rows and adapters hold."""
    p = make(48, 130, 256, 16, 6, 7)
    ids = np.arange(48) % 6
    want = check(p, ids)
    p["A"][2] = float("inf")
    p["B"][2] = float("nan")
    p["A"][4, 3, 7] = float("nan")
    p["x"][ids == 2] = float("nan")
    p["base"][ids == 4] = float("inf")
    got = dg.dg_lora_bf16(*(p[n].to(DEV) for n in ("x", "A", "B")), torch.from_numpy(ids).int().to(DEV),
                          p["base"].to(DEV), scales=p["scales"].to(DEV))
    keep = torch.from_numpy((ids != 2) & (ids != 4)).to(DEV)
    assert torch.equal(want[keep], got[keep])
    # and a row alone gives what it gives in the batch
    for t in (0, 17, 47):
        one = dg.dg_lora_bf16(p["x"][t:t + 1].to(DEV), p["A"].to(DEV), p["B"].to(DEV),
                              torch.from_numpy(ids[t:t + 1]).int().to(DEV), p["base"][t:t + 1].to(DEV),
                              scales=p["scales"].to(DEV))
        if ids[t] not in (2, 4):
            d = (one[0].float() - got[t].float()).abs()
            assert (d <= 2.0 ** -7 * got[t].float().abs() + 1e-3).all()


@pytest.mark.parametrize("ldx,ldb,ldo,offset", [(264, 104, 112, 0), (256, 101, 103, 0), (256, 104, 104, 1),
                                                (512, 200, 104, 4)])
def test_strides_and_untouched_columns(ldx, ldb, ldo, offset):
    p = make(21, 100, 256, 16, 4, 8)
    ids = ids_of(21, 4, "mixed")
    want = check(p, ids)
    x, base = strided(p["x"], ldx), strided(p["base"], ldb, offset)
    buf = torch.full((21 * ldo + offset + ldo,), 5.0, dtype=BF, device=DEV)
    out = buf[offset:].as_strided((21, 100), (ldo, 1))
    dg.dg_lora_bf16(x, p["A"].to(DEV), p["B"].to(DEV), torch.from_numpy(ids).int().to(DEV), base, out,
                    scales=p["scales"].to(DEV))
    assert torch.equal(out, want)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[offset:].as_strided((21, 100), (ldo, 1)).fill_(False)
    assert (buf[rest] == 5.0).all()


def test_in_place():
    p = make(37, 96, 256, 16, 4, 9)
    ids = ids_of(37, 4, "mixed")
    want = check(p, ids)
    y = p["base"].to(DEV)
    got = dg.dg_lora_bf16(p["x"].to(DEV), p["A"].to(DEV), p["B"].to(DEV), torch.from_numpy(ids).int().to(DEV),
                          y, y, scales=p["scales"].to(DEV))
    assert got is y and torch.equal(y, want)


def test_empty():
    p = make(0, 16, 128, 8, 2, 1)
    assert dg.dg_lora_bf16(p["x"].to(DEV), p["A"].to(DEV), p["B"].to(DEV),
                           torch.empty(0, dtype=torch.int32, device=DEV)).shape == (0, 16)
    p = make(3, 0, 128, 8, 2, 1)
    assert dg.dg_lora_bf16(p["x"].to(DEV), p["A"].to(DEV), p["B"].to(DEV),
                           torch.zeros(3, dtype=torch.int32, device=DEV)).shape == (3, 0)


def test_offsets_past_32_bits():
    """Adapters past 2^31 elements of A and B, rows of x and out past 2^32 bytes."""
    L, rank, K, N, T = 70, 128, 128, 1 << 18, 5
    A = torch.empty(L, rank, K, dtype=BF, device=DEV)
    B = torch.empty(L, N, rank, dtype=BF, device=DEV)
    assert B.numel() > 1 << 31
    p = make(T, 32, K, rank, 1, 10)
    A[L - 1] = p["A"][0].to(DEV)
    B[L - 1].zero_()
    B[L - 1, -32:] = p["B"][0].to(DEV)
    far = 1 << 30
    x = torch.empty(far * (T - 1) + K, dtype=BF, device=DEV).as_strided((T, K), (far, 1))
    x.copy_(p["x"])
    ids = torch.full((T,), L - 1, dtype=torch.int32, device=DEV)
    got = dg.dg_lora_bf16(x, A, B, ids)
    torch.cuda.synchronize()
    ref, size = R.lora(host(p["x"]), host(p["A"]), host(p["B"]), np.zeros(T, int), None, None, None)
    g = host(got[:, -32:]).astype(np.float64)
    assert np.all(np.abs(g - ref) <= R.lora_tolerance(ref, size, K))
    assert (got[:, :-32] == 0).all()


def test_same_bits_other_stream_and_graph():
    p = make(64, 192, 2048, 16, 16, 11)
    ids = torch.from_numpy(ids_of(64, 16, "mixed")).int().to(DEV)
    x, A, B, base, scales = (p[n].to(DEV) for n in ("x", "A", "B", "base", "scales"))
    want = dg.dg_lora_bf16(x, A, B, ids, base, scales=scales)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dg.dg_lora_bf16(x, A, B, ids, base, scales=scales, stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    out = torch.empty_like(base)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dg.dg_lora_bf16(x, A, B, ids, base, out, scales=scales)
    for r in range(4):
        out.zero_()
        dg.dg_lora_bf16(x[:5], A, B, ids[:5], scales=scales)       # eager work in between
        if r == 2:                                             # new rows for the same graph
            ids.copy_(ids.flip(0))
            want = dg.dg_lora_bf16(x, A, B, ids, base, scales=scales)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_beside_the_fp8_projection():
    """base = dg_gemm_fp8_nt of the quantised activations, the adapters from the bf16 ones."""
    p = make(64, 256, 512, 16, 8, 12)
    rng = np.random.default_rng(0)
    W = bf(rng, 256, 512, scale=0.05).to(DEV)
    x = p["x"].to(DEV)
    wq, ws = dg.dg_quantize_fp8_128x128(W)
    xq, xs = dg.dg_quantize_fp8_1x128(x)
    y = dg.dg_gemm_fp8_nt(xq, xs, wq, ws)
    p["base"] = y.cpu()
    check(p, ids_of(64, 8, "mixed"))


def test_refusals():
    p = {n: v.to(DEV) for n, v in make(8, 32, 256, 16, 2, 13).items()}
    ids = torch.zeros(8, dtype=torch.int32, device=DEV)
    x, A, B = p["x"], p["A"], p["B"]
    with pytest.raises(dg.DGError):                       # K % 128
        dg.dg_lora_bf16(x[:, :200].contiguous(), A[:, :, :200].contiguous(), B, ids)
    with pytest.raises(dg.DGError):                       # R % 8
        dg.dg_lora_bf16(x, A[:, :12].contiguous(), B[:, :, :12].contiguous(), ids)
    with pytest.raises(dg.DGError):                       # row stride of x
        dg.dg_lora_bf16(strided(x, 260), A, B, ids)
    with pytest.raises(dg.DGError):                       # alignment of x
        dg.dg_lora_bf16(strided(x, 256, offset=1), A, B, ids)
    with pytest.raises(TypeError):
        dg.dg_lora_bf16(x.float(), A, B, ids)
    with pytest.raises(TypeError):
        dg.dg_lora_bf16(x, A, B, ids.long())
    with pytest.raises(ValueError):
        dg.dg_lora_bf16(x, A, B[:, :, :8].contiguous(), ids)
    with pytest.raises(ValueError):
        dg.dg_lora_bf16(x, A, B, ids[:4])
    with pytest.raises(ValueError):
        dg.dg_lora_bf16(x, A.transpose(0, 1).contiguous().transpose(0, 1), B, ids)
    with pytest.raises(dg.DGError):                       # a batch that needs a workspace
        dg.dg_lora_bf16(x.repeat(30, 1), A, B, ids.repeat(30),
                        workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
