"""A stack of feed-forward layers on a residual stream, in 8 bits: trained with gated_ffn, and run a
few tokens at a time from weights that are quantised once.

    stream = stream + out                    (the layer before's)
    out = w2 (act(gate norm(stream)) * up norm(stream))

    python examples/feed_forward.py          # needs an MI355X
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402


class FeedForward(torch.nn.Module):
    def __init__(self, K, N, device, seed=0):
        super().__init__()
        g = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.norm = torch.nn.Parameter(1 + 0.1 * n(K))
        self.w13 = torch.nn.Parameter((n(2 * N, K) * K ** -0.5).bfloat16())
        self.w2 = torch.nn.Parameter((n(K, N) * N ** -0.5).bfloat16())

    def forward(self, x, stream):
        """x T x K bfloat16, the layer before's output; returns this one's and the stream."""
        out, h = dg.gated_ffn(x, self.w13, self.w2, residual=stream, norm_weight=self.norm)
        return out, x if h is None else h


class Stack(torch.nn.Module):
    def __init__(self, layers, K, N, device="cuda:0"):
        super().__init__()
        self.layers = torch.nn.ModuleList(FeedForward(K, N, device, i) for i in range(layers))

    def forward(self, x):
        stream = None
        for layer in self.layers:
            x, stream = layer(x, stream)
        return x + stream

    @torch.no_grad()
    def packed(self):
        """Codes and scales of the weights, for decode()."""
        return [(layer.norm.detach(), *dg.dg_quantize_fp8_128x128(layer.w13), *dg.dg_quantize_fp8_128x128(layer.w2))
                for layer in self.layers]


def decode(packed, x):
    """The stack's output for a few tokens x (T x K bfloat16): three calls a layer, no readback, so
    a step can be captured."""
    stream = None
    for norm, b13, s13, b2, s2 in packed:
        q, s, h, _, _ = dg.dg_rms_norm_fp8(x, norm, residual=stream)
        a, sa, _, _ = dg.dg_gated_fp8_nt(q, s, b13, s13)
        x, stream = dg.dg_gemm_fp8_nt(a, sa, b2, s2), h
    return x + stream


def main(T=200, K=512, N=384):
    stack = Stack(2, K, N)
    g = torch.Generator(device="cuda:0").manual_seed(9)
    x = torch.randn(T, K, generator=g, device="cuda:0").bfloat16()
    target = torch.randn(T, K, generator=g, device="cuda:0")
    opt = torch.optim.SGD(stack.parameters(), lr=0.1)
    for step in range(3):
        opt.zero_grad()
        loss = (stack(x).float() - target).square().mean()
        loss.backward()
        opt.step()
        print(f"step {step}: loss {float(loss.detach()):.4f}", flush=True)
    packed = stack.packed()
    with torch.no_grad():
        same = torch.equal(decode(packed, x[:16]), stack(x[:16]))
    print(f"16 tokens decoded, as the stack computes them: {same}", flush=True)
    assert same and bool(loss.isfinite())


if __name__ == "__main__":
    main()
