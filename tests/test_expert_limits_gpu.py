"""The expert-layer operators at the borders of their sizes, where a launch, a
workspace or an index changes its form, and on inputs that are valid but seldom."""
import math

import pytest
import torch

import matrix_orthogonalizing_optimizer_muon_amd as M
import test_experts_gpu as base
from oracle import experts_oracle as O

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


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("live", [0, 100000, -5])
def test_combine_backward_clears_rows_that_slots_name(dtype, live):
    """Rows from offsets[E] on are zero although slots name them, in whatever order their waves run: the last choices
    have the first rows here."""
    tokens, k, cols = 100000, 2, 24
    n = tokens * k
    y, dout = (torch.randn(r, cols, generator=gen(2)).to(dtype).cuda() for r in (n, tokens))
    slots = torch.arange(n, dtype=I, device="cuda").flip(0).view(tokens, k).contiguous()
    w = torch.rand(tokens, k, generator=gen(3)).cuda() + 0.5
    off = torch.tensor([0, 7, live], dtype=I, device="cuda")
    base.poison((n, cols), dtype)
    dy, dw = M.combine_backward(dout, y, slots, w, off)
    want = (w[..., None] * dout.float()[:, None]).view(n, cols).flip(0)
    want[max(live, 0):] = 0
    assert (dy[max(live, 0):] == 0).all()
    # one product rounded to fp32 and to the type
    base.close(dy, want.cpu().double(), (base.HALF[dtype] + base.ULP) * want.abs().cpu().double(), "dy")
    dots = (y.flip(0).view(tokens, k, cols).double() * dout[:, None].double())
    base.close(dw, dots.sum(2).cpu(), cols * base.ULP * dots.abs().sum(2).cpu(), "dweights")


# rows of the experts, outer, inner: few rows, tiles through registers, large bf16 tiles, odd k
@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("sizes", [([3, 2], 40, 256), ([3, 2], 33, 37), ([1], 8, 1600), ([700, 900], 259, 515),
                                   ([600, 900], 776, 512)])
def test_a_row_that_names_no_token_is_a_row_of_zeros(dtype, sizes):
    """Whichever kernel takes the product: zero, and NaN where the matrix has an infinity."""
    counts, outer, inner = sizes
    x, w, _, rows, off = base.product_inputs(counts, outer, inner, dtype, True, 2, 4)
    rows[0], rows[counts[0] - 1] = x.shape[0], -9
    w[0, 3, 1], w[0, 7, inner - 1], w[-1, 5, inner // 2] = math.inf, -math.inf, math.nan
    o = torch.tensor(off, dtype=I, device="cuda")
    base.poison((rows.shape[0], outer), dtype)
    y = M.grouped_matmul(x.cuda(), w.cuda(), o, rows=rows.cuda()).cpu().double()
    want = O.matmul(x, w, off, rows)
    fine = torch.isfinite(want)
    assert not fine[0, 3] and not fine[0, 7] and (want[0][fine[0]] == 0).all()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(y[torch.isinf(want)], want[torch.isinf(want)])
    z = torch.where(torch.isfinite(w), w, torch.zeros((), dtype=dtype))
    bound = base.HALF[dtype] * want.abs() + inner * base.ULP * O.matmul(x.abs(), z.abs(), off, rows) + base.TINY[dtype]
    assert ((y - want).abs()[fine] <= bound[fine]).all()
