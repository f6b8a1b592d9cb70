"""Grouped feed-forward calls without the number of groups, which none of them can tell.  Looked at
on the CPU: the check is the first."""
import pytest

torch = pytest.importorskip("torch")

import moe_grouped_gemm_lhs_amd as dg  # noqa: E402


def test_gated_backward_asks_for_the_number_of_groups():
    """Without it rows of every group but the first would be left as they were."""
    dh, gu, sgu = torch.zeros(4, 128), torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    idx = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="group_idx needs groups"):
        dg.dg_gated_backward(dh, gu, sgu, group_idx=idx)
    for groups in ({}, dict(groups=3), dict(group_idx=idx, groups=3)):       # the next check's turn
        with pytest.raises(ValueError, match="must be on a GPU"):
            dg.dg_gated_backward(dh, gu, sgu, **groups)


def test_weight_gradients_ask_for_the_number_of_groups():
    """Without it the sum over all rows, whatever their groups, would be returned."""
    p, sp = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 1)
    idx = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="groups must be a number"):
        dg.dg_grouped_wgrad_fp8_contiguous(p, sp, p, sp, idx, None)
    with pytest.raises(ValueError, match="must be on a GPU"):
        dg.dg_grouped_wgrad_fp8_contiguous(p, sp, p, sp, idx, 2)
