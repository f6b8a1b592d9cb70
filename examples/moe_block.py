"""A mixture-of-experts block with per-request adapters, put together from this package's
calls: the shared FP8 projection with the requests' low-rank adapters beside it, the gate,
and the routed experts' grouped FP8 projections.

    out[t] = shared(x[t]) + adapter_{request of t}(x[t]) + sum_j w[t, j] expert_{id[t, j]}(x[t])

`prefill` lays the chosen rows out in the contiguous form (segments aligned to 128 rows) and
gives the balance loss, differentiable by the gate's weight; `decode` uses the masked form,
whose masked_m is the gate's counts.  Neither reads anything back to the host.

    python examples/moe_block.py        # needs an MI355X
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402

ALIGN = 128


@dataclass
class MoeBlock:
    gate: torch.Tensor            # E x K float32
    shared: tuple                 # codes N x K and scales of the shared projection
    experts: tuple                # codes E x N x K and scales
    A: torch.Tensor               # L x R x K bfloat16
    B: torch.Tensor               # L x N x R bfloat16
    scales: torch.Tensor          # L float32
    k: int = 2
    balance: float = 1e-2

    def _beside(self, x, xq, xs, adapter):
        y = dg.dg_gemm_fp8_nt(xq, xs, *self.shared)
        return dg.dg_lora_bf16(x, self.A, self.B, adapter, y, y, scales=self.scales)

    def prefill(self, x, adapter, valid=None):
        """x T x K bfloat16, adapter T int32 (-1: none), valid T bool (False: padding).
        Returns out (T x N float32), the experts' counts and the balance loss."""
        T, K = x.shape
        E = self.gate.shape[0]
        xq, xs = dg.dg_quantize_fp8_1x128(x)
        y = self._beside(x, xq, xs, adapter)
        ids, w, counts, loss = dg.moe_route(x.float() @ self.gate.t(), self.k, row_valid=valid,
                                            normalize=True, balance=self.balance)
        # rows of the contiguous form: each expert's segment, then one spare row for choices
        # that are none; its length is bounded by sizes that the host knows
        seg = (counts + ALIGN - 1) // ALIGN * ALIGN
        end = seg.cumsum(0)
        rows = -(-(T * self.k + E * (ALIGN - 1) + 1) // ALIGN) * ALIGN
        at = self._places(ids, counts, end - seg, rows - 1)
        group = torch.searchsorted(end, torch.arange(rows, device=x.device), right=True).int()
        group = torch.where(group < E, group, -1)
        token = torch.arange(T * self.k, device=x.device) // self.k
        a = torch.zeros(rows, K, dtype=torch.uint8, device=x.device)
        sa = torch.zeros(rows, K // 128, device=x.device)
        a[at] = xq.view(torch.uint8)[token]
        sa[at] = xs[token]
        c = dg.dg_grouped_gemm_fp8_contiguous(a, sa, *self.experts, group)
        return self._combine(y, c, at, w), counts, loss

    def decode(self, x, adapter):
        """One token of each of T requests.  Returns out (T x N float32) and the counts."""
        T, K = x.shape
        E = self.gate.shape[0]
        xq, xs = dg.dg_quantize_fp8_1x128(x)
        y = self._beside(x, xq, xs, adapter)
        ids, w, counts, _, _ = dg.dg_moe_route(x.float() @ self.gate.t(), self.k, normalize=True,
                                               count=True)
        # each expert has room for every request, and a row more for choices that are none
        first = torch.arange(E, device=x.device) * T
        at = self._places(ids, counts, first, E * T)
        token = torch.arange(T * self.k, device=x.device) // self.k
        a = torch.zeros(E * T + 1, K, dtype=torch.uint8, device=x.device)
        sa = torch.zeros(E * T + 1, K // 128, device=x.device)
        a[at] = xq.view(torch.uint8)[token]
        sa[at] = xs[token]
        c = dg.dg_grouped_gemm_fp8_masked(a[:-1].view(E, T, K), sa[:-1].view(E, T, -1), *self.experts,
                                          counts)
        c = torch.cat([c.view(E * T, -1), c.new_zeros(1, c.shape[-1])])
        return self._combine(y, c, at, w), counts

    @staticmethod
    def _places(ids, counts, first, spare):
        """Row of each choice: its expert's first row plus its place among the expert's
        choices, in the order of rows; `spare` for -1."""
        flat = ids.reshape(-1).long()
        order = torch.sort(flat, stable=True).indices
        none = (flat < 0).sum()
        before = counts.cumsum(0) - counts
        place = torch.empty_like(flat)
        place[order] = torch.arange(flat.numel(), device=flat.device) - none
        e = flat.clamp_min(0)
        return torch.where(flat >= 0, first[e] + place - before[e], spare)

    @staticmethod
    def _combine(y, c, at, w):
        T, k = w.shape
        # a choice that is none has weight 0, and its spare row may hold anything
        rows = torch.where(w[..., None] != 0, c[at].view(T, k, -1).float(), 0.0)
        return y.float() + (w[..., None] * rows).sum(1)


def make(E=16, N=512, K=1024, L=6, R=16, k=2, seed=0, device="cuda"):
    """A block of random weights."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return scale * torch.randn(*shape, generator=g, device=device)

    shared = dg.dg_quantize_fp8_128x128(normal(N, K, scale=K ** -0.5))
    pairs = [dg.dg_quantize_fp8_128x128(normal(N, K, scale=K ** -0.5)) for _ in range(E)]
    # one stack of bytes: float8 tensors have no stack
    experts = (torch.stack([q.view(torch.uint8) for q, _ in pairs]), torch.stack([s for _, s in pairs]))
    return MoeBlock(normal(E, K, scale=K ** -0.5), shared, experts,
                    normal(L, R, K, scale=K ** -0.5).bfloat16(), normal(L, N, R, scale=0.1).bfloat16(),
                    torch.full((L,), 2.0, device=device), k=k)


def main():
    block = make()
    block.gate.requires_grad_()
    opt = torch.optim.SGD([block.gate], lr=0.5)
    x = torch.randn(1000, 1024, device="cuda").bfloat16() + 0.5
    adapter = (torch.arange(1000, device="cuda") // 150).int() - 1       # prompts; the first has none
    valid = torch.arange(1000, device="cuda") < 960                      # the rest is padding
    for step in range(5):
        opt.zero_grad()
        out, counts, loss = block.prefill(x, adapter, valid)
        loss.backward()
        opt.step()
        print(f"step {step}: balance loss {float(loss.detach()):.5f}, busiest expert {int(counts.max())} of "
              f"{int(counts.sum())} choices", flush=True)
    with torch.no_grad():
        out, counts = block.decode(x[:32], adapter[:32])
    print(f"decode: out {tuple(out.shape)}, {int(counts.sum())} choices over "
          f"{int((counts > 0).sum())} experts", flush=True)


if __name__ == "__main__":
    main()
