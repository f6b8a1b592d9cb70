"""Calls on a stream that is not the current one, while that one is busy: what a call allocates
for itself is not written by work that the current stream has still to do."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16


def calls():
    """Each call without its outputs, and the sizes in bytes of what it allocates."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    G, cap, N, K = 4, 64, 256, 512
    a, sa = dg.dg_quantize_fp8_1x128(normal(G * cap, K))
    pairs = [dg.dg_quantize_fp8_128x128(normal(N, K)) for _ in range(G)]
    b = torch.stack([q.view(torch.uint8) for q, _ in pairs])
    sb = torch.stack([s for _, s in pairs])
    a = a.view(torch.uint8)
    masked_m = torch.tensor([64, 3, 0, 17], dtype=torch.int32, device=DEV)
    a2, sa2 = a.repeat(2, 1)[:512], sa.repeat(2, 1)[:512]
    group = torch.arange(512, device=DEV).div(128, rounding_mode="floor").int()
    group[500:] = -1
    z = normal(3000, 64)
    ids = (torch.arange(300, device=DEV) % 3).int()
    x, A, B = normal(300, K).to(BF), normal(3, 16, K).to(BF), normal(3, N, 16).to(BF)
    route = dg.dg_moe_route(z, 4, balance=1.0)
    gw = normal(3000, 4)
    return {
        "dense": lambda **k: (dg.dg_gemm_fp8_nt(a, sa, b[0], sb[0], **k),),
        "contiguous": lambda **k: (dg.dg_grouped_gemm_fp8_contiguous(a2, sa2, b, sb, group, **k),),
        "masked": lambda **k: (dg.dg_grouped_gemm_fp8_masked(a.view(G, cap, K), sa.view(G, cap, -1), b, sb,
                                                             masked_m, **k),),
        "route": lambda **k: dg.dg_moe_route(z, 4, balance=1.0, **k),
        "backward": lambda **k: (dg.dg_moe_route_backward(z, route[0], grad_weights=gw, coef=route[4], **k),),
        "lora": lambda **k: (dg.dg_lora_bf16(x, A, B, ids, **k),),
    }


def test_outputs_of_a_side_stream_are_its_own():
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=DEV)
    for name, f in calls().items():
        print(f"[case] {name} on a side stream", flush=True)
        want = f()
        torch.cuda.synchronize()
        # the current stream: work of some milliseconds, then writes to blocks that it has given
        # back, of the sizes that the outputs take
        for _ in range(6):
            big @ big
        for t in want:
            torch.empty_like(t).fill_(7)
        got = f(stream=side)
        torch.cuda.synchronize()
        for w, h in zip(want, got):
            assert torch.equal(w, h), name
        del want, got
