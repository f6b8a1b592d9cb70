"""examples/moe_block.py: the gate, the adapters and the FP8 calls as they are used together,
against the same block in 64 bits from the same codes and weights; the balance loss's
gradient through the gate's weight; the example's own run."""
import importlib.util
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
moe_block = importlib.util.module_from_spec(spec)
sys.modules["moe_block"] = moe_block
spec.loader.exec_module(moe_block)


def values(codes, scales, block_rows):
    """The numbers that codes and block scales stand for, in 64 bits on the CPU."""
    q = codes.cpu().view(torch.uint8).view(torch.float8_e4m3fn).double()
    s = scales.cpu().double().repeat_interleave(128, -1)
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, -2)
    return q * s[..., :q.shape[-2], :q.shape[-1]]


def reference(block, x, adapter, ids, w):
    xq, xs = dg.dg_quantize_fp8_1x128(x)
    xv = values(xq, xs, 1)
    out = xv @ values(*block.shared, 128).t()
    size = xv.abs() @ values(*block.shared, 128).abs().t()
    xb = x.cpu().double()
    for i in range(block.A.shape[0]):
        r = adapter.cpu() == i
        out[r] += float(block.scales[i]) * (xb[r] @ block.A[i].cpu().double().t()) @ block.B[i].cpu().double().t()
    experts = values(*block.experts, 128)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e >= 0:
                out[t] += float(w[t, j]) * (experts[e] @ xv[t])
    return out, size


def check(out, block, x, adapter, ids, w):
    want, size = reference(block, x, adapter, ids, w)
    # two bf16 roundings of the shared part, one of each expert's; fp32 sums of K = 1024 terms
    tol = 3 * 2.0 ** -8 * (want.abs().max() + 1) + size.max() * 2.0 ** -14
    assert (out.cpu().double() - want).abs().max() <= tol


@pytest.fixture(scope="module")
def block():
    return moe_block.make()


def test_prefill(block):
    T = 200
    x = torch.randn(T, 1024, device="cuda").bfloat16()
    adapter = (torch.arange(T, device="cuda") // 30).int() - 1
    valid = torch.arange(T, device="cuda") % 9 != 0
    out, counts, loss = block.prefill(x, adapter, valid)
    ids, w, n, l, _ = dg.dg_moe_route(x.float() @ block.gate.t(), block.k, row_valid=valid, normalize=True,
                                      balance=block.balance)
    assert torch.equal(n, counts) and torch.equal(l, loss)
    assert int(counts.sum()) == block.k * int(valid.sum())
    check(out, block, x, adapter, ids.cpu(), w.cpu())


@pytest.mark.parametrize("T", [1, 17, 64])
def test_decode(block, T):
    x = torch.randn(T, 1024, device="cuda").bfloat16()
    adapter = torch.randint(-1, 6, (T,), device="cuda").int()
    out, counts = block.decode(x, adapter)
    ids, w, n, _, _ = dg.dg_moe_route(x.float() @ block.gate.t(), block.k, normalize=True, count=True)
    assert torch.equal(n, counts)
    check(out, block, x, adapter, ids.cpu(), w.cpu())


def test_balance_loss_trains_the_gate(block):
    """The gate's gradient is the loss's by the logits through the product with x."""
    x = torch.randn(300, 1024, device="cuda").bfloat16()
    adapter = torch.full((300,), -1, dtype=torch.int32, device="cuda")
    gate = block.gate.clone().requires_grad_()
    trained = moe_block.MoeBlock(gate, block.shared, block.experts, block.A, block.B, block.scales)
    _, counts, loss = trained.prefill(x, adapter)
    loss.backward()
    xd, gd = x.cpu().double(), block.gate.cpu().double().requires_grad_()
    p = torch.softmax(xd @ gd.t(), 1)
    f = counts.cpu().double() * 16 / (2 * 300)
    want = 1e-2 * (f * p.mean(0)).sum()
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) <= 1e-4 * float(want.detach())
    # logits rounded to fp32, gradients in fp32, a product of 300 terms
    assert (gate.grad.cpu().double() - gd.grad).norm() <= 1e-4 * gd.grad.norm()


def test_main(capsys):
    moe_block.main()
    printed = capsys.readouterr().out
    assert "step 4" in printed and "decode" in printed
