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


# ------------------------------------- more threads than a launch takes along one axis (2^32)

def rand(*shape, seed, dtype=F):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def spots(n, at):
    """Rows at both ends and around `at`."""
    return torch.cat([torch.arange(max(0, m - 2000), min(n, m + 2000), device="cuda") for m in (0, n // 2, at, n)]).unique()


def test_combine_backward_of_2_to_26_choices():
    n = (1 << 26) + 5
    y, dout = rand(n, 1, seed=5, dtype=B), rand(n, 1, seed=6, dtype=B)
    w = rand(n, 1, seed=7)
    slots = torch.arange(n, dtype=I, device="cuda").flip(0).view(n, 1).contiguous()
    off = torch.tensor([0, n - 3], dtype=I, device="cuda")
    base.poison((n, 1), B)
    dy, dw = M.combine_backward(dout, y, slots, w, off)
    want = (w * dout.float()).to(B).flip(0)       # one product each, rounded alike
    want[n - 3:] = 0
    assert torch.equal(dy, want)
    assert torch.equal(dw, y.flip(0).float() * dout.float())


def test_route_of_2_to_28_tokens():
    n = (1 << 28) + 70
    l = rand(n, 2, seed=8, dtype=B)
    r = M.route(l, 1)
    second = l[:, 1] > l[:, 0]
    assert torch.equal(r.experts[:, 0], second.to(I))
    assert (r.weights == 1).all()
    first = n - int(second.sum())
    assert r.offsets.tolist() == [0, first, n]
    assert torch.equal(r.rows[:first], (~second).nonzero()[:, 0].to(I))
    assert torch.equal(r.rows[first:], second.nonzero()[:, 0].to(I))
    assert torch.equal(r.slots[r.rows.long(), 0], torch.arange(n, dtype=I, device="cuda"))
    # and the gradient, 16 lanes a token
    r = M.route(l, 1, normalize=False)
    dw = rand(n, 1, seed=9)
    base.poison((n, 2), B)
    d = M.route_backward(dw, l, r, normalize=False)
    assert torch.isfinite(d).all()
    at = spots(n, (1 << 28) // 64 * 64)
    ids, lc = r.experts[at, 0].tolist(), l[at].cpu()
    p = torch.softmax(lc.double(), 1)
    hot = torch.nn.functional.one_hot(torch.tensor(ids), 2).double()
    up = (p * hot * dw[at].cpu().double()).sum(1, keepdim=True)
    # exp of a difference below 2^4 rounded to fp32, a sum of two, a quotient; then products of two such
    tol = (2 ** 4 + 2 + 8) * base.ULP
    want = hot * up - p * up
    base.close(d[at], want, base.HALF[B] * want.abs() + 2 * tol * (hot + p) * up.abs() + 2.0 ** -120, "logits' gradient")


def test_route_backward_of_2_to_26_tokens_a_wave_each():
    n, k = (1 << 26) + 9, 17
    chosen = torch.arange(k, dtype=I, device="cuda").repeat(n, 1)
    w = torch.full((n, k), 1 / 32, device="cuda")
    dw = rand(n, k, seed=10)
    l = torch.zeros(n, k, dtype=B, device="cuda")
    r = M.Routing(w, chosen, chosen, chosen.view(-1), chosen[0])
    base.poison((n, k), B)
    d = M.route_backward(dw, l, r)
    assert torch.isfinite(d).all()
    at = spots(n, 1 << 26)
    x = dw[at].cpu().double() / 32                  # exact
    # 17 terms, and a product and a difference
    want = x - x.sum(1, keepdim=True) / 32
    size = x.abs() + x.abs().sum(1, keepdim=True) / 32
    base.close(d[at], want, base.HALF[B] * want.abs() + 20 * base.ULP * size, "logits' gradient")


@pytest.mark.parametrize("grad", [False, True])
def test_rows_products_of_2_to_30_rows(grad):
    n = (1 << 30) + 70
    x = rand(n, 1, seed=11)
    w = torch.tensor([[[1.7]]], device="cuda")
    o = torch.tensor([0, n - 3], dtype=I, device="cuda")
    y = M.grouped_input_grad(x, w, o) if grad else M.grouped_matmul(x, w, o)
    assert (y[-3:] == 0).all()
    assert torch.equal(y[:-3], x[:-3] * w[0])       # one product each


def test_weight_grad_of_2_to_24_tiles():
    experts, cols = 1024, (1 << 20) + 1
    dy, x = rand(3, 1, seed=12), rand(3, cols, seed=13)
    o = torch.tensor([0] * 513 + [3] * 512, dtype=I, device="cuda")
    dw = M.grouped_weight_grad(dy, x, o)
    assert (dw[:512] == 0).all() and (dw[513:] == 0).all()
    want = (dy.double() * x.double()).sum(0).cpu()
    size = (dy.double() * x.double()).abs().sum(0).cpu()
    base.close(dw[512, 0], want, base.HALF[F] * want.abs() + 3 * base.ULP * size, "dw")


@pytest.mark.parametrize("grad", [False, True])
def test_few_rows_of_2_to_24_columns(grad):
    experts, cols = 64, (1 << 24) - 1
    w = rand(experts, cols, seed=14, dtype=B)
    x = rand(experts, 1, seed=15, dtype=B)
    o = torch.arange(experts + 1, dtype=I, device="cuda")
    if grad:
        y = M.grouped_input_grad(x, w.view(experts, 1, cols), o)
    else:
        y = M.grouped_matmul(x, w.view(experts, cols, 1), o)
    assert torch.equal(y, (x.float() * w.float()).to(B))   # one product each


def test_gated_of_2_to_29_rows_without_a_checkpoint():
    """More rows than a checkpoint of them could have (its blocks of one column pair): none is asked for."""
    n = (1 << 29) + 8
    gu = rand(n, 2, seed=16, dtype=B)
    base.poison((n, 1), B)
    h = M.gated(gu)
    assert torch.isfinite(h).all()
    at = spots(n, 1 << 29)
    want = O.gated(gu[at].cpu())
    base.close(h[at], want, base.HALF[B] * want.abs() + 24 * base.ULP * want.abs() + 2.0 ** -120, "h")
    with pytest.raises(M.MuonError, match="groups of 8 columns"):
        M.gated(gu, checkpoint="int8")


def test_parameters_under_no_grad():
    x, w, _, rows, off = base.product_inputs([3, 0, 9], 24, 40, B, True, 0, 17)
    o, wd = torch.tensor(off, dtype=I, device="cuda"), w.cuda()
    p = torch.nn.Parameter(wd)
    with pytest.raises(ValueError, match="w requires grad"):
        M.grouped_matmul(x.cuda(), p, o, rows=rows.cuda())
    with torch.no_grad():
        y = M.grouped_matmul(x.cuda(), p, o, rows=rows.cuda())
    assert torch.equal(y, M.grouped_matmul(x.cuda(), wd, o, rows=rows.cuda()))


@pytest.mark.parametrize("tokens,experts,k", [(32768, 64, 8), (32769, 64, 8), (16384, 128, 3), (16385, 128, 3),
                                              (20000, 129, 2), (65536, 256, 8), (65537, 300, 4), (65536, 1024, 2),
                                              (32768, 3, 2), (32769, 3, 2), (65, 129, 17)])
def test_route_on_both_sides_of_its_scan(tokens, experts, k):
    l = rand(tokens, experts, seed=18)
    l[::7, experts // 2] = -math.inf
    r = M.route(l, k)
    _, ids = torch.sort(l, dim=1, descending=True, stable=True)
    ids = ids[:, :k].contiguous()
    order = torch.argsort(ids.reshape(-1), stable=True)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(tokens * k, device="cuda")
    assert torch.equal(r.experts.long(), ids)
    assert torch.equal(r.rows.long(), order // k)
    assert torch.equal(r.slots.long().reshape(-1), slots)
    counts = torch.bincount(ids.reshape(-1), minlength=experts).cumsum(0)
    assert r.offsets.tolist() == [0] + counts.tolist()


@pytest.mark.parametrize("off", [1, 8])
@pytest.mark.parametrize("gather", [False, True])
def test_weight_grad_of_many_small_matrices(off, gather):
    """Few tiles of long sums and more than 96 large ones, on 16 bytes (8 elements past) and off them."""
    counts = [130 + 3 * (e % 40) for e in range(128)]
    x, _, dy, rows, offsets = base.product_inputs(counts, 128, 120, B, gather, 0, 19)
    base.poison((128, 128, 120), B)
    dw = M.grouped_weight_grad(base.guarded(dy, off), base.guarded(x, off), torch.tensor(offsets, dtype=I, device="cuda"),
                               rows=rows.cuda() if gather else None)
    want = O.weight_grad(dy, x, offsets, rows)
    size = O.weight_grad(dy.abs(), x.abs(), offsets, rows)
    base.close(dw, want, base.HALF[B] * want.abs() + max(counts) * base.ULP * size, "dw")


# ------------------------------------------------------------- operands past 2^31 bytes and elements

def test_products_that_gather_from_2_to_30_elements():
    """More than the large tiles' 31-bit lane offsets hold: the tiles staged through registers take them."""
    inner, outer, experts, x_rows = 1024, 512, 64, (1 << 20) + 8
    x = torch.zeros(x_rows, inner, dtype=B, device="cuda")
    tail = rand(300, inner, seed=20, dtype=B)
    x[-300:] = tail
    x[:300] = tail.flip(0)
    n = 3000
    g = gen(21)
    pick = torch.randint(0, 600, (n,), generator=g)
    rows = torch.where(pick < 300, pick, pick - 600 + x_rows).to(I)
    far = torch.where(pick < 300, 299 - pick, pick - 300)           # the row of `tail` that a row names
    off = [n * e // experts for e in range(experts + 1)]
    o = torch.tensor(off, dtype=I, device="cuda")
    w = rand(experts, outer, inner, seed=22, dtype=B)
    dy = rand(n, outer, seed=23, dtype=B)
    near = tail.cpu()[far]
    base.poison((n, outer), B)
    y = M.grouped_matmul(x, w, o, rows=rows.cuda())
    want = O.matmul(near, w.cpu(), off)
    base.close(y, want, base.HALF[B] * want.abs() + inner * base.ULP * O.matmul(near.abs(), w.cpu().abs(), off), "matmul")
    base.poison((experts, outer, inner), B)
    dw = M.grouped_weight_grad(dy, x, o, rows=rows.cuda())
    want = O.weight_grad(dy.cpu(), near, off)
    size = O.weight_grad(dy.cpu().abs(), near.abs(), off)
    base.close(dw, want, base.HALF[B] * want.abs() + 47 * base.ULP * size, "dw")


def test_weight_grad_by_large_tiles_of_2_to_31_elements():
    inner, outer, experts, n = 2048, 16, 16, (1 << 20) + 40         # 128 large tiles
    x = torch.zeros(n, inner, dtype=B, device="cuda")
    dy = torch.zeros(n, outer, dtype=B, device="cuda")
    for t, seed in ((x, 24), (dy, 25)):
        t[-300:] = rand(300, t.shape[1], seed=seed, dtype=B)
        t[:100] = rand(100, t.shape[1], seed=seed + 2, dtype=B)
    off = [e * (n // experts) for e in range(experts)] + [n]
    off[-2] = n - 200
    o = torch.tensor(off, dtype=I, device="cuda")
    base.poison((experts, outer, inner), B)
    dw = M.grouped_weight_grad(dy, x, o)
    assert (dw[1:-2] == 0).all()
    for e, part in ((0, slice(0, 100)), (-2, slice(n - 300, n - 200)), (-1, slice(n - 200, n))):
        a, b = dy[part].cpu().double(), x[part].cpu().double()
        want, size = a.t() @ b, a.abs().t() @ b.abs()
        base.close(dw[e], want, base.HALF[B] * want.abs() + 200 * base.ULP * size, f"dw of {e}")
