"""The kernels that a product grouped by expert can take, each at sizes that reach
it, against the fp64 oracle with the bounds of test_experts_gpu.py (one rounding
of the result, K accumulation steps); the router's kernels by width; and the
example that runs the layer."""
import importlib.util
import math
import os

import pytest
import torch

import matrix_orthogonalizing_optimizer_muon_amd as M
import test_experts_gpu as base
from oracle import experts_oracle as O

pytestmark = pytest.mark.gpu

F, B, I = torch.float32, torch.bfloat16, torch.int32
gen = base.gen

# rows of the experts, outer, inner: past 4 rows an expert in bf16 (16 in fp32) and 1280 strips, so that the
# tile kernels take them
TILES = {
    "cuts of a row tile": ([300, 128, 129, 256, 511, 1, 0, 640, 384], 520, 776),
    "last columns of 128 and less": ([1500, 700], 896, 640),
    "more experts than lanes": ([100 + 37 * (e % 5) - (100 if e % 11 == 3 else 0) for e in range(70)], 264, 520),
    "five hundred experts": ([9 + e % 30 for e in range(500)], 72, 136),
    "one k tile and less": ([900, 1200, 600], 1032, 8),
    "few long k": ([700, 40], 2048, 1544),
}


@pytest.mark.parametrize("name", list(TILES))
@pytest.mark.parametrize("gather", [False, True])
def test_large_tiles(name, gather):
    counts, outer, inner = TILES[name]
    x, w, dy, rows, off = base.product_inputs(counts, outer, inner, B, gather, 300 if gather else 0, 90)
    if gather:
        rows[5], rows[len(rows) // 2] = x.shape[0], -3        # read as rows of zeros
    aligned(x, w, dy, rows, off)


def aligned(x, w, dy, rows, off):
    """base.check_products on tensors that start on 16 bytes."""
    keep, base.guarded = base.guarded, lambda t, off=8: keep(t, off)
    try:
        return base.check_products(x, w, dy, rows, off)
    finally:
        base.guarded = keep


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("gather", [False, True])
def test_small_tiles(dtype, gather):
    """Odd sides: no 16-byte rows, so the tiles staged through registers."""
    base.check_products(*base.product_inputs([2000, 0, 700, 41], 259, 515, dtype, gather, 70 if gather else 0, 91))


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("sides", [(16, 8), (17, 32), (31, 33), (48, 64), (100, 31), (64, 129), (65, 127), (33, 4)])
def test_few_rows(dtype, sides):
    """Strips that end inside 16 columns, k that ends inside a step or a chunk, 0 to 33 rows an expert."""
    for gather in (False, True):
        base.check_products(*base.product_inputs([1, 0, 2, 15, 16, 17, 33, 0, 1], *sides, dtype, gather, 2, 92))


def test_few_rows_of_many_experts():
    base.check_products(*base.product_inputs([e % 3 for e in range(200)], 72, 520, B, True, 4, 93))
    base.check_products(*base.product_inputs([e % 2 for e in range(1024)], 40, 24, F, False, 0, 94))


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sides", [(40, 72), (129, 33)])
def test_weight_grad_in_parts(dtype, gather, sides):
    """Few tiles and long sums: experts' rows in parts, some of them empty."""
    base.check_products(*base.product_inputs([5000, 0, 2500, 3], *sides, dtype, gather, 9 if gather else 0, 99))
    base.check_products(*base.product_inputs([1, 129, 6000], *sides, dtype, gather, 0, 100))


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_weight_grad_in_parts_from_a_checkpoint(dtype, kind):
    x, _, dy, rows, off = base.product_inputs([3000, 0, 1700], 72, 70, dtype, True, 4, 101)
    c = M.checkpoint(x.cuda(), kind)
    back = M.restore(c).cpu()
    base.poison((3, 72, 70), dtype)
    dw = M.grouped_weight_grad(dy.cuda(), c, torch.tensor(off, dtype=I, device="cuda"), rows=rows.cuda())
    want = O.weight_grad(dy, back, off, rows)
    size = O.weight_grad(dy.abs(), back.abs(), off, rows)
    base.close(dw, want, base.HALF[dtype] * want.abs() + 3000 * base.ULP * size + base.TINY[dtype], "in parts")


@pytest.mark.parametrize("off", [[0, 1900, 600, 2500], [-7, -3, 1200, 1100], [50, 900, 1500, 2 ** 31 - 1],
                                 [9, 0, 0, 0], [0, 2 ** 31 - 1, 3, 150]])
def test_large_tiles_of_broken_offsets(off):
    x, w, dy, rows, _ = base.product_inputs([900, 1200, 700], 520, 264, B, True, 0, 95)
    aligned(x, w, dy, rows, off)


def test_large_tiles_keep_infinities_in_their_rows():
    x, w, dy, _, off = base.product_inputs([600, 900], 512, 776, B, False, 0, 96)
    x[4, 2], x[1490, 775], dy[130, 3], dy[700, 511] = math.inf, math.nan, -math.inf, math.nan
    o = torch.tensor(off, dtype=I, device="cuda")
    y = M.grouped_matmul(x.cuda(), w.cuda(), o).cpu()
    dx = M.grouped_input_grad(dy.cuda(), w.cuda(), o).cpu()
    dw = M.grouped_weight_grad(dy.cuda(), x.cuda(), o).cpu()
    assert (~torch.isfinite(y)).any(1).nonzero().flatten().tolist() == [4, 1490]
    assert (~torch.isfinite(dx)).any(1).nonzero().flatten().tolist() == [130, 700]
    want = torch.zeros(dw.shape, dtype=torch.bool)
    want[0, :, 2] = want[1, :, 775] = want[0, 3] = want[1, 511] = True
    assert torch.equal(~torch.isfinite(dw), want)


def test_rows_alone_give_what_they_give_in_a_batch():
    """A row's product does not depend on its neighbours beyond the order of the
    sum: the kernels for few rows against the large tiles."""
    x, w, _, _, off = base.product_inputs([600, 900, 800], 1024, 776, B, False, 0, 97)
    wd = w.cuda()
    y = M.grouped_matmul(x.cuda(), wd, torch.tensor(off, dtype=I, device="cuda")).cpu().double()
    at = [0, 599, 600, 1499, 1500, 2299]
    few = M.grouped_matmul(x[at].cuda(), wd, torch.tensor([0, 2, 4, 6], dtype=I, device="cuda")).cpu().double()
    size = O.matmul(x[at].abs(), w.abs(), [0, 2, 4, 6])
    # each is off by its rounding and 776 accumulation steps
    assert ((few - y[at]).abs() <= 2 * base.HALF[B] * y[at].abs() * (1 + 2 ** -7) + 2 * 776 * base.ULP * size).all()


@pytest.mark.parametrize("kind", ["none", "int8"])
def test_large_layer_in_a_graph(kind):
    """Large tiles in a captured layer, replayed on new inputs, bit for bit the eager result."""
    def one(a):
        if kind == "none":
            x, wgu, wd, logits, dout = a
            r = M.route(logits, 4)
            gu = M.grouped_matmul(x, wgu, r.offsets, rows=r.rows)
            h = M.gated(gu)
            y = M.grouped_matmul(h, wd, r.offsets)
            dy, dwt = M.combine_backward(dout, y, r.slots, r.weights, r.offsets)
            dgu, hb = M.gated_backward(M.grouped_input_grad(dy, wd, r.offsets), gu)
            return [M.combine(y, r.slots, r.weights), M.grouped_weight_grad(dy, hb, r.offsets),
                    M.grouped_weight_grad(dgu, x, r.offsets, rows=r.rows), M.grouped_input_grad(dgu, wgu, r.offsets)]
        return base.layer(*a, 4, kind)

    def inputs(seed):
        return base.layer_inputs(B, tokens=1500, seed=seed, d=768, f=512, experts=8)
    a = inputs(100)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        one(a)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = one(a)
    for seed in range(101, 105):
        new = inputs(seed)
        for t, v in zip(a, new):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = one(new)
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("shape", [(70, 2, 2), (66, 16, 16), (130, 17, 16), (66, 17, 17), (100, 128, 16), (100, 129, 3),
                                   (64, 256, 16), (65, 257, 16), (1, 256, 1)])
def test_route_by_width(dtype, normalize, shape):
    """Both forms of the router (up to 256 experts and 16 choices, and beyond)."""
    base.test_route_and_its_gradient(dtype, normalize, shape)


def test_route_at_the_border_of_its_scan():
    """65536 tokens are the most whose counts the placing blocks add up by themselves."""
    for tokens in (65535, 65536, 65537):
        l = torch.randn(tokens, 5, generator=gen(98))
        l[::7, 2] = -math.inf
        r = M.route(l.cuda(), 2)
        _, ids = torch.sort(l, dim=1, descending=True, stable=True)
        ids = ids[:, :2].contiguous()
        order = torch.argsort(ids.reshape(-1), stable=True)
        assert torch.equal(r.experts.cpu().long(), ids)
        assert torch.equal(r.rows.cpu().long(), order // 2)
        assert r.offsets.tolist() == [0] + torch.bincount(ids.reshape(-1), minlength=5).cumsum(0).tolist()


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("keep", ["none", "int8", "e4m3"])
def test_example_trains(keep):
    losses, _, _ = example().train(steps=30, keep=keep)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.6 * losses[0], losses
