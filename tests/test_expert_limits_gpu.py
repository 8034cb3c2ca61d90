"""The expert-layer operators at the borders of their sizes, where a launch, a
workspace or an index changes its form, and on inputs that are valid but seldom."""
import pytest
import torch

import matrix_orthogonalizing_optimizer_muon_amd as M
import test_experts_gpu as base

pytestmark = pytest.mark.gpu

F, B, I = torch.float32, torch.bfloat16, torch.int32
gen = base.gen


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_weight_grad_of_no_rows_from_a_checkpoint(dtype, kind):
    c = M.checkpoint(torch.randn(37, 72, generator=gen(1)).to(dtype).cuda(), kind)
    dy = torch.empty(0, 24, dtype=dtype, device="cuda")
    rows = torch.empty(0, dtype=I, device="cuda")
    base.poison((3, 24, 72), dtype)
    dw = M.grouped_weight_grad(dy, c, torch.zeros(4, dtype=I, device="cuda"), rows=rows)
    assert dw.shape == (3, 24, 72) and (dw == 0).all()
