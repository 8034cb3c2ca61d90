"""The vocabulary operators at the borders of what they take, on inputs that are
valid but seldom: few rows that count in a long call, logits far from zero, w at any
address.  Bounds as in test_vocabulary_gpu.py."""
import math

import pytest
import torch

import matrix_orthogonalizing_optimizer_muon_amd as M
import test_vocabulary_gpu as base
from oracle import vocabulary_oracle as O

pytestmark = pytest.mark.gpu

F, B = torch.float32, torch.bfloat16
HALF, TINY, ULP = base.HALF, base.TINY, base.ULP
inf = math.inf


def on_gpu(values):
    return [None if t is None else t.cuda() for t in values]


def gradients(dloss, x, w, ids, teacher, tau, lse=None):
    """(dx, dw) of a loss call with gradients, or of one from lse."""
    if teacher is None:
        return M.classifier_loss_grads(dloss, x, w, ids)[2:] if lse is None else \
            M.classifier_loss_backward(dloss, x, w, ids, lse)
    kw = {"temperature": tau}
    return M.distill_loss_grads(dloss, x, w, teacher, ids, **kw)[2:] if lse is None else \
        M.distill_loss_backward(dloss, x, w, teacher, ids, lse, **kw)


def check_gradients(x, w, dloss, ids, teacher, tau, what, twice):
    """Both forms on these inputs (on the GPU) against the oracle there.  twice: dl is kept to twice its digits."""
    if teacher is None:
        at, q = O.target_weights(ids, w.shape[0])
        arg = torch.zeros(x.shape[0], dtype=torch.float64, device="cuda")
    else:
        at, q = O.teacher_weights(teacher, ids, w.shape[0], tau)
        t = torch.where(at >= 0, teacher.double(), math.nan)
        arg = torch.nan_to_num((t.nan_to_num(-inf).max(1).values - t.nan_to_num(inf).min(1).values) / tau, posinf=0,
                               neginf=0)
    half = HALF[x.dtype]
    lse = O.loss(x, w, at, q, tau)[1].float()
    for form in ("both", "backward"):
        # two roundings to the type where exponentials come first; twice: the rest's, and nine bits of a fraction
        rounding = half * half + 2.0 ** -10 if twice else half * (1 + half) * (2 if form == "both" else 1)
        bounds = base.bounds_of(x, w, dloss, at, q, arg, tau, rounding)[2:]
        given = lse if form == "backward" else None
        base.poison(tuple(x.shape), tuple(w.shape))
        got, want = gradients(dloss, x, w, ids, teacher, tau, given), O.grads(dloss, x, w, at, q, tau, given)
        for name, g, v, b in zip(("dx", "dw"), got, want, bounds):
            base.close(g, v, b + half * (v.abs() + b) + TINY[x.dtype], f"{what}: {form} {name}")


# ------------------------------------------------ few rows count in a long call

def few_live(tokens, vocab, dim, live, where, dtype, k, seed):
    """Inputs of which `live` rows count: spread over the call, or its last ones."""
    x, w, dloss, ids, teacher = base.inputs(tokens, vocab, dim, dtype, k, seed, absent=0.0)
    keep = torch.randperm(tokens, generator=base.gen(seed))[:live] if where == "spread" else \
        torch.arange(tokens - live, tokens)
    dead = torch.ones(tokens, dtype=torch.bool)
    dead[keep] = False
    ids[dead] = -1
    return on_gpu((x, w, dloss, ids, teacher))


@pytest.mark.parametrize("where", ["spread", "last"])
@pytest.mark.parametrize("k,tau", [(0, 1.0), (3, 2.0)])
@pytest.mark.parametrize("dtype", [B, F], ids=str)
@pytest.mark.parametrize("tokens,vocab,dim,live", [
    (8192, 1000, 256, 820), (2048, 4000, 256, 200), (1024, 1000, 256, 65), (1024, 1000, 256, 100),
    (1024, 1000, 256, 128), (1024, 1000, 256, 129), (8192, 2048, 1024, 500), (20000, 300, 96, 1), (20000, 300, 96, 64),
    (20000, 300, 96, 65), (20000, 300, 96, 128), (20000, 300, 96, 200), (20000, 300, 96, 513), (20000, 300, 96, 2240),
    (20000, 300, 96, 2241), (8193, 40, 8, 900)])
def test_few_rows_of_many_count(tokens, vocab, dim, live, dtype, k, tau, where):
    """dw's sum is cut into parts by the rows of the call, of which those that count may leave a part one k-tile
    or none."""
    x, w, dloss, ids, teacher = few_live(tokens, vocab, dim, live, where, dtype, k, tokens + live)
    check_gradients(x, w, dloss, ids, teacher, tau, where, twice=False)


def test_a_short_last_chunk():
    """32768 rows of this vocabulary are a chunk, and a chunk's dw two parts; the last chunk has two k-tiles."""
    x, w, dloss, ids, _ = on_gpu(base.inputs(32768 + 100, 32768, 64, B, 0, 5, absent=0.0))
    at, q = O.target_weights(ids, 32768)
    _, _, dx, dw = M.classifier_loss_grads(dloss, x, w, ids)
    arg = torch.zeros(x.shape[0], dtype=torch.float64, device="cuda")
    bound = base.bounds_of(x, w, dloss, at, q, arg, 1.0, HALF[B] * (1 + HALF[B]) * 2)[2:]
    for name, g, v, b in zip(("dx", "dw"), (dx, dw), O.grads(dloss, x, w, at, q), bound):
        base.close(g, v, b + HALF[B] * (v.abs() + b) + TINY[B], name)


# ------------------------------------------------------------ logits far from zero

@pytest.mark.parametrize("k,tau", [(0, 1.0), (5, 2.0)])
@pytest.mark.parametrize("dtype", [B, F], ids=str)
@pytest.mark.parametrize("tokens,vocab", [(20, 5001), (100, 6001), (300, 1000), (300, 2050), (700, 129)])
@pytest.mark.parametrize("shift", [-700.0, 700.0])
def test_all_logits_far_from_zero(tokens, vocab, dtype, shift, k, tau):
    """exp of a whole row's logits under- or overflows; a vocabulary that ends inside a slab."""
    dim = 64
    x, w, dloss, ids, teacher = base.inputs(tokens, vocab, dim, dtype, k, tokens + vocab)
    x = (1 + 0.1 * x.float()).to(dtype)
    w = (w.float() + shift / dim).to(dtype)
    check_gradients(*on_gpu((x, w, dloss, ids, teacher)), tau, f"shift {shift}", twice=dtype == B and tokens <= 128)


@pytest.mark.parametrize("dtype", [B, F], ids=str)
@pytest.mark.parametrize("tokens,vocab", [(20, 5001), (100, 6001), (300, 2050)])
def test_a_slab_of_logits_of_minus_infinity(tokens, vocab, dtype):
    """Columns whose logits overflow to -inf are those of probability zero, as where they are merely large."""
    dim = 64
    x, w, dloss, ids, _ = base.inputs(tokens, vocab, dim, dtype, 0, tokens)
    w = (w.float() - 700.0 / dim).to(dtype)
    x = (1 + 0.1 * x.float()).to(dtype)
    w[:, 0] = 0
    x[:, 0] = 2.0 ** 66
    ids[(ids >= 64) & (ids < 192)] = 3
    got = []
    for size in (2.0 ** 40, 2.0 ** 66):     # logits of -2^106, and -2^132
        w[64:192, 0] = -size
        got.append(M.classifier_loss_grads(*on_gpu((dloss, x, w, ids))))
    assert all(bool(t.isfinite().all()) for t in got[0])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("tau", [1.0, 2.0 ** -20])
@pytest.mark.parametrize("dtype", [B, F], ids=str)
@pytest.mark.parametrize("tokens,vocab", [(20, 5001), (100, 6001), (300, 2050)])
def test_exponents_of_more_than_24_bits(tokens, vocab, dtype, tau):
    """Logits over the temperature of 2^25, where whole numbers of fp32 lie 4 apart: one entry has all of its row's
    probability.  It and the target's entry of dl are dloss, rounded twice to bf16 at the most."""
    g = base.gen(tokens)
    x, w = torch.zeros(tokens, 8), torch.randn(vocab, 8, generator=g)
    x[:, 0] = (4096 + 32 * torch.randint(0, 128, (tokens,), generator=g)) * tau
    w[:, 0] = 4096.0 + 32 * torch.randint(0, 31, (vocab,), generator=g)
    w[vocab // 3, 0] = 4096.0 + 32 * 32
    x, w = x.to(dtype), w.to(dtype)
    ids = torch.randint(0, vocab, (tokens, 1), generator=g)
    dloss, teacher = torch.randn(tokens, generator=g), torch.zeros(tokens, 1)
    x, w, ids, dloss, teacher = on_gpu((x, w, ids, dloss, teacher))
    loss, lse, dx, dw = M.distill_loss_grads(dloss, x, w, teacher, ids, temperature=tau)
    at, q = O.target_weights(ids[:, 0], vocab)
    z = x.double() @ w.double().t() / tau
    want_loss, want_lse = O.loss(x, w, at, q, tau)
    size = z.abs().max(1).values * 16 * ULP
    base.close(lse, want_lse, size, "lse")
    base.close(loss, want_loss, size * tau * tau + want_loss * 16 * ULP, "loss")
    want = O.grads(dloss, x, w, at, q, tau)
    # entries of dl, and what a probability and a weight of one are off by where they cancel
    soft = torch.zeros_like(z).scatter_add_(1, at.clamp_min(0), q)
    dl = O.logits_grad(dloss, x, w, at, q, tau).abs() * (2 * HALF[dtype] + 2.0 ** -10 if dtype == B else 32 * ULP)
    dl += 16 * ULP * tau * dloss.double().abs()[:, None] * (torch.exp(z - want_lse[:, None]) + soft)
    for got, v, s in ((dx, want[0], dl @ w.double().abs()), (dw, want[1], dl.t() @ x.double().abs())):
        base.close(got, v, s + (HALF[dtype] + 8 * ULP) * (v.abs() + s) + TINY[dtype], "gradient")


@pytest.mark.parametrize("tau", [1.0, 0.7, 2.3])
@pytest.mark.parametrize("dtype", [B, F], ids=str)
@pytest.mark.parametrize("tokens,vocab", [(20, 5001), (100, 6001), (300, 2050)])
def test_slabs_of_logits_far_below_the_others(tokens, vocab, dtype, tau):
    """Columns of probability zero are that at whatever size of their logits, from -2^17 down to fp32's lowest and below
    it: nothing else moves by a bit."""
    dim, g = 64, base.gen(tokens)
    x, w, dloss, ids, teacher = base.inputs(tokens, vocab, dim, dtype, 3, tokens)
    w[:, 0] = 0
    x[:, 0] = 2.0 ** 66 * (1 + torch.rand(tokens, generator=g)).to(dtype)
    ids[(ids >= 64) & (ids < 256)] = 3
    size = (1 + torch.rand(192, generator=g)).to(dtype)
    got = []
    for e in (-49, -40, -31, -20, 0, 30, 60, 61, 62):
        w[64:256, 0] = -(size.float() * 2.0 ** e).to(dtype)
        args = on_gpu((dloss, x, w, teacher, ids))
        got.append((*M.distill_loss_grads(*args, temperature=tau), *M.distill_loss(*args[1:], temperature=tau)))
        assert all(bool(t.isfinite().all()) for t in got[-1]), f"2^{e}"
        assert all(torch.equal(a, b) for a, b in zip(got[0], got[-1])), f"2^{e}"


# ---------------------------------------------------------------- w at any address

@pytest.mark.parametrize("k,tau", [(0, 1.0), (5, 2.0)])
@pytest.mark.parametrize("tokens,vocab,dim", [(1, 300, 72), (5, 33, 8), (31, 515, 2104), (64, 777, 1096), (65, 777, 1096),
                                              (100, 5003, 72), (128, 300, 72), (127, 516, 135)])
def test_few_rows_keep_their_digits_wherever_w_lies(tokens, vocab, dim, k, tau):
    x, w, dloss, ids, teacher = on_gpu(base.inputs(tokens, vocab, dim, B, k, tokens + dim))
    for off in (1, 3, 4):
        check_gradients(x, base.guarded(w, off), dloss, ids, teacher, tau, f"w {off} elements on", twice=True)


@pytest.mark.parametrize("tokens", [1, 50, 100])
def test_few_rows_keep_their_digits_in_a_vocabulary_of_2_to_the_21(tokens):
    x, w, dloss, ids, teacher = on_gpu(base.inputs(tokens, (1 << 21) + 5, 9, B, 3, tokens, absent=0.0))
    check_gradients(x, w, dloss, ids, teacher, 1.5, "vocabulary of 2^21 and more", twice=True)


@pytest.mark.parametrize("form", ["both", "backward"])
@pytest.mark.parametrize("tokens,vocab", [(300, 1024), (500, 1000), (300, (1 << 21) + 64)])
def test_equal_dloss_is_not_rounded_wherever_w_lies(tokens, vocab, form):
    """test_equal_dloss_is_not_rounded's w, off its alignment, in a small vocabulary (whose logits are kept), and in one
    that the large tiles do not address: others' entries of dl are dloss / vocab, rounded as a power of two (none) or
    as 1 / 1000 is (by 2^-9 at the most)."""
    d, g = 40, 1.0036 / 256
    x = torch.randn(tokens, d, generator=base.gen(1)).bfloat16().cuda()
    w = base.guarded(torch.zeros(vocab, d).bfloat16())
    targets = torch.randperm(vocab, generator=base.gen(2))[:tokens].cuda()
    dloss = torch.full((tokens,), g).cuda()
    lse = torch.full((tokens,), math.log(vocab)).cuda() if form == "backward" else None
    dw = gradients(dloss, x, w, targets, None, 1.0, lse)[1]
    at, q = O.target_weights(targets, vocab)
    want = O.grads(dloss, x, w, at, q, 1.0, lse)[1]
    rows = x.double().abs()
    own = torch.zeros(vocab, d, dtype=torch.float64, device="cuda").index_add_(0, targets, rows * g)
    p = 1 / vocab
    near = 0.0 if math.log2(vocab).is_integer() else abs(p / float(torch.tensor(p).bfloat16()) - 1) + 2.0 ** -10
    # a target's entry, 1 - p, may be off by its distance to one or half a step; lse of 14 by half a step, 2^-21
    slack = max(2.0 ** -10, p) * own + (tokens + 32) * ULP * own + (near + (tokens + 64) * ULP) * rows.sum(0) * g * p
    base.close(dw, want, slack + HALF[B] * (want.abs() + slack), "dw")


@pytest.mark.parametrize("tokens,vocab", [(8192 + 321, 131072), (600, (1 << 21) + 5)])
def test_chunks_wherever_w_lies(tokens, vocab):
    """One unit for the dloss of all chunks, whose dw goes on from one to the next."""
    x, w, dloss, ids, _ = on_gpu(base.inputs(tokens, vocab, 16, B, 0, 23, absent=0.05))
    dloss[:400] *= 2.0 ** -8
    check_gradients(x, base.guarded(w), dloss, ids, None, 1.0, "chunks", twice=False)


@pytest.mark.parametrize("sizes", [(300, 500, 128), (400, 2100, 136), (20, 500, 64), (100, 5000, 72)])
def test_a_step_in_a_graph_with_w_off_alignment(sizes):
    """Captured once, replayed on other values and numbers of rows that count, with eager work between."""
    args = list(base.step_inputs(2, B, *sizes))
    args[3] = base.guarded(args[3])
    base.model_step(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = base.model_step(*args)
    for seed in (3, 4, 5):
        for a, b in zip(args, base.step_inputs(seed, B, *sizes)):
            a.copy_(b)
        args[1][seed * 3:] = -1          # targets: few are left
        want = base.model_step(*args)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


# ----------------------------------------------------- operands that 31 bits do not address

@pytest.mark.parametrize("dtype", [B, F], ids=str)
@pytest.mark.parametrize("tokens,vocab,dim", [
    (3, 300, (1 << 21) + 9), (1000, 600, (1 << 21) + 8), (20, (1 << 21) - 8, 1032), (70, (1 << 21) - 8, 1032),
    (70, (1 << 21) + 3, 1032), ((1 << 20) + 70, 40, 2056)])
def test_long_operands(tokens, vocab, dim, dtype):
    """x or w of 2^31 elements and more, and widths and vocabularies past 2^21.  64 columns are not zero, the first and
    last among them: sums over the others are exact, so that the bounds are those of 64 columns."""
    x, w, dloss, ids, _ = base.inputs(tokens, vocab, 64, dtype, 0, 7, absent=0.02)
    x, w, dloss, ids = on_gpu((x, w, dloss, ids))
    cols = torch.cat([torch.tensor([0, dim - 1]), 1 + torch.randperm(dim - 2, generator=base.gen(8))[:62]]).cuda()
    at, q = O.target_weights(ids, vocab)
    arg = torch.zeros(tokens, dtype=torch.float64, device="cuda")
    half = HALF[dtype]
    rounding = half * half + 2.0 ** -10 if dtype == B and tokens <= 128 else half * (1 + half) * 2
    bounds = base.bounds_of(x, w, dloss, at, q, arg, 1.0, rounding)
    want = (*O.loss(x, w, at, q), *O.grads(dloss, x, w, at, q))
    wide = [torch.zeros(t.shape[0], dim, dtype=dtype, device="cuda") for t in (x, w)]
    for t, narrow in zip(wide, (x, w)):
        t[:, cols] = narrow
    loss, lse = M.classifier_loss(*wide, ids)
    got = M.classifier_loss_grads(dloss, *wide, ids)
    back = M.classifier_loss_backward(dloss, *wide, ids, want[1].float())
    from_lse = O.grads(dloss, x, w, at, q, 1.0, want[1].float())
    for values, name in (((loss, lse), "loss"), (got[:2], "loss with gradients")):
        for g, v, b in zip(values, want, bounds):
            base.close(g, v, b, name)
    for pair, wanted in ((got[2:], want[2:]), (back, from_lse)):
        for g, v, b, name in zip(pair, wanted, bounds[2:], ("dx", "dw")):
            base.close(g[:, cols], v, b + half * (v.abs() + b) + TINY[dtype], name)
            assert int(torch.count_nonzero(g)) == int(torch.count_nonzero(g[:, cols])), f"{name}: other columns"


@pytest.mark.parametrize("dtype", [B, F], ids=str)
def test_embedding_of_a_long_table(dtype):
    """Rows past 2^31 elements of the table, of its gradient and of the outputs; whole numbers, exactly."""
    vocab, dim, n = (1 << 21) + 3, 1032, 3000
    t = torch.cat([torch.tensor([vocab - 1, vocab, 0, -1]), torch.randint(vocab - 100, vocab, (n - 4,),
                                                                        generator=base.gen(1))]).cuda()
    table = torch.zeros(vocab, dim, dtype=dtype, device="cuda")
    table[-100:] = torch.randint(-8, 9, (100, dim), generator=base.gen(2)).to(dtype).cuda()
    out = M.embed(t, table)
    named = (t >= 0) & (t < vocab)
    assert torch.equal(out, torch.where(named[:, None], table[torch.where(named, t, 0)], 0.0))
    dout = torch.randint(-2, 3, (n, dim), generator=base.gen(3)).to(dtype).cuda()
    dtable = M.embed_backward(dout, t, vocab)
    low = vocab - 100
    want = torch.zeros(100, dim, dtype=torch.float64, device="cuda")
    here = (t >= low) & (t < vocab)
    want.index_add_(0, t[here] - low, dout[here].double())
    assert torch.equal(dtable[low:].double(), want)
    assert torch.equal(dtable[0].double(), dout[2].double()) and not dtable[1:low].any()
