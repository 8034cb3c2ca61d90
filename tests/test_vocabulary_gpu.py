"""The vocabulary operators against the fp64 oracle.

Tolerances are bounds, not fits.  A result rounded to a type is off by at most
half a step, torch.finfo(type).eps / 2 of the value (bf16 2^-8, fp32 2^-24).  A
sum of K products or terms accumulated in fp32 in any order, each step within one
unit in the last place (2^-23), is off by at most K 2^-23 times the sum of the
terms' magnitudes.  bounds_of() counts the operations of the losses."""
import math

import pytest
import torch

import matrix_orthogonalizing_optimizer_muon_amd as M
from oracle import vocabulary_oracle as O

pytestmark = pytest.mark.gpu

F, B, I, J = torch.float32, torch.bfloat16, torch.int32, torch.int64
HALF = {t: torch.finfo(t).eps / 2 for t in (F, B)}
ULP = 2.0 ** -23
TINY = {F: 2.0 ** -149, B: 2.0 ** -133}
inf, nan = math.inf, math.nan


def gen(seed):
    return torch.Generator().manual_seed(seed)


def guarded(t, off=1):
    """t on the GPU inside a larger allocation of NaN (whole numbers: of names of nothing),
    starting off elements past its alignment."""
    n = t.numel()
    big = torch.full((n + 2 * off + 64,), nan if t.is_floating_point() else -77, dtype=t.dtype, device="cuda")
    v = big[off:off + n].view(t.shape)
    v.copy_(t)
    return v


def poison(*tensors):
    """Leaves NaN in the memory that the next allocations of these sizes take, so that an
    output left unwritten shows."""
    for t in tensors:
        torch.empty(t, device="cuda").fill_(nan)
    torch.cuda.synchronize()


def close(got, want, bound, what):
    got, want = got.cpu().double(), want.cpu().double()
    bad = ~((got - want).abs() <= bound.cpu())
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}: " \
                          f"{got[bad][0]} for {want[bad][0]}"


# ------------------------------------------------------------------- embedding

EMBED = [(1, 1, 1), (1, 1000, 64), (3, 7, 33), (64, 5, 520), (65, 5, 8), (200, 300, 136), (1000, 3, 17),
         (1025, 40000, 24), (777, 129, 1031), (4099, 513, 512), (20000, 700, 8), (300, 140000, 16)]


def tokens_of(n, vocab, seed, index=J, absent=0.1):
    """Uneven tokens: half of them among a few, some that name nothing."""
    g = gen(seed)
    t = torch.randint(0, vocab, (n,), generator=g)
    few = torch.randint(0, min(vocab, 3), (n,), generator=g)
    t = torch.where(torch.rand(n, generator=g) < 0.5, few, t)
    bad = torch.tensor([-1, vocab, -100, vocab + 5, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 6, (n,), generator=g)]
    return torch.where(torch.rand(n, generator=g) < absent, bad, t).to(index)


@pytest.mark.parametrize("index", [I, J], ids=str)
@pytest.mark.parametrize("dtype", [F, B], ids=str)
@pytest.mark.parametrize("n,vocab,dim", EMBED)
def test_embed(n, vocab, dim, dtype, index):
    t = tokens_of(n, vocab, n + dim, index)
    table = torch.randn(vocab, dim, generator=gen(dim)).to(dtype)
    for off, scale in ((0, 1.0), (1, 45.25)):
        poison((n, dim))
        got = M.embed(guarded(t, off), guarded(table, off), scale=scale)
        want = O.embed(t, table, scale)
        close(got, want, want.abs() * (HALF[dtype] + 2 * ULP) + TINY[dtype], "out")
        assert got.dtype == dtype


@pytest.mark.parametrize("index", [I, J], ids=str)
@pytest.mark.parametrize("dtype", [F, B], ids=str)
@pytest.mark.parametrize("n,vocab,dim", EMBED)
def test_embed_backward(n, vocab, dim, dtype, index):
    t = tokens_of(n, vocab, n + vocab, index)
    dout = torch.randn(n, dim, generator=gen(vocab)).to(dtype)
    at = O.named(t, vocab)
    count = torch.zeros(vocab + 1).index_add_(0, torch.where(at < 0, vocab, at), torch.ones(n))[:vocab, None].double()
    for off, scale in ((0, 1.0), (1, 45.25)):
        poison((vocab, dim))
        got = M.embed_backward(guarded(dout, off), guarded(t, off), vocab, scale=scale)
        want = O.embed_backward(dout, t, vocab, scale)
        summed = O.embed_backward(dout.abs(), t, vocab, scale) * (count + 2) * ULP
        close(got, want, summed + HALF[dtype] * (want.abs() + summed) + TINY[dtype], "dtable")


@pytest.mark.parametrize("word", [0, 37, 299])
@pytest.mark.parametrize("n", [31, 32, 33, 63, 64, 65, 128, 129, 1000, 5000])
def test_embed_backward_of_one_token(n, word):
    """All places hold one token: its row is joined from windows, whole numbers exactly."""
    t = torch.full((n,), word)
    dout = torch.randint(-8, 9, (n, 40), generator=gen(n)).float()
    want = O.embed_backward(dout, t, 300)
    assert torch.equal(M.embed_backward(dout.cuda(), t.cuda(), 300).cpu().double(), want)


def test_embed_backward_of_long_rows_side_by_side():
    """Rows of 33 and more places whose ends and starts share windows, whole numbers exactly."""
    counts = [65, 1, 66, 200, 0, 64, 33, 129, 3, 63, 70, 32, 34, 31, 0, 33, 2, 300]
    t = torch.cat([torch.full((c,), v) for v, c in enumerate(counts)])
    t = t[torch.randperm(t.shape[0], generator=gen(5))]
    dout = torch.randint(-8, 9, (t.shape[0], 24), generator=gen(6)).float()
    assert torch.equal(M.embed_backward(dout.cuda(), t.cuda(), 18).cpu().double(), O.embed_backward(dout, t, 18))


def test_embed_backward_repeats_its_bits():
    t = tokens_of(3000, 500, 1).cuda()
    dout = torch.randn(3000, 128, generator=gen(2)).cuda()
    first = M.embed_backward(dout, t, 500)
    assert all(torch.equal(first, M.embed_backward(dout, t, 500)) for _ in range(5))


def test_embed_passes_values_on():
    """Infinities and NaN of named rows arrive, those of others do not."""
    table = torch.tensor([[inf, -inf, nan, 1.0], [2.0, 2.0, 2.0, 2.0]]).cuda()
    out = M.embed(torch.tensor([0, 5, 1]).cuda(), table).cpu()
    assert out[0, 0] == inf and out[0, 1] == -inf and out[0, 2].isnan() and out[0, 3] == 1
    assert torch.equal(out[1:], torch.tensor([[0.0] * 4, [2.0] * 4]))
    d = M.embed_backward(table[:, :2].contiguous(), torch.tensor([-1, 1]).cuda(), 3).cpu()
    assert torch.equal(d, torch.tensor([[0.0, 0.0], [2.0, 2.0], [0.0, 0.0]]))


# ---------------------------------------------------------------------- losses

SIZES = [(1, 1, 1), (1, 16, 16), (1, 1000, 64), (5, 33, 7), (17, 129, 200), (64, 128, 64), (130, 300, 72),
         (257, 515, 129), (300, 1024, 256), (513, 70, 520), (700, 1111, 264), (520, 2050, 128), (385, 6007, 136),
         (129, 129, 8), (2100, 40, 16), (16, 5003, 136), (33, 40000, 72), (64, 777, 1096), (65, 777, 1096),
         (48, 4096, 333), (64, 4097, 72), (31, 515, 2100), (128, 300, 72), (127, 515, 136), (97, 2050, 264),
         (100, 5003, 72), (64, 8192, 1144), (20, 16383, 2264)]


def inputs(tokens, vocab, dim, dtype, k, seed, absent=0.2, index=J):
    """Logits of standard deviation 4, so that a row's sum is that of a few entries, which
    lie anywhere; targets may come twice in a row."""
    g = gen(seed)
    x = torch.randn(tokens, dim, generator=g).to(dtype)
    w = (torch.randn(vocab, dim, generator=g) * (4 / math.sqrt(dim))).to(dtype)
    dloss = torch.randn(tokens, generator=g)
    ids = torch.randint(0, vocab, (tokens, max(1, k)), generator=g)
    bad = torch.tensor([-1, vocab, -100, 2 ** 31 - 1])[torch.randint(0, 4, ids.shape, generator=g)]
    gone = torch.rand(ids.shape, generator=g) < absent
    gone |= torch.rand(tokens, 1, generator=g) < absent if tokens > 1 else torch.zeros(1, 1, dtype=torch.bool)
    ids = torch.where(gone, bad, ids).to(index)
    teacher = 3 * torch.randn(tokens, max(1, k), generator=g)
    return x, w, dloss, (ids if k else ids[:, 0].contiguous()), (teacher if k else None)


def bounds_of(x, w, dloss, at, q, arg, tau, rounding):
    """Elementwise bounds of (loss, lse, dx, dw) by the operations behind them:
    a logit is a sum of dim products; an exponent of it is scaled, has a largest one taken off twice and is raised
    (four roundings of at most its size, one step of the result); lse is a sum of vocab terms and a logarithm;
    q's exponents are differences of teacher logits over tau (arg: the largest), three roundings, summed over k;
    an entry of dl is rounded to the type of x, off by `rounding` of its value; dx and dw are sums of vocab and of rows products."""
    xd, wd = x.double(), w.double()
    vocab, dim, k = w.shape[0], w.shape[1], at.shape[1]
    z = xd @ wd.t() / tau
    dz = xd.abs() @ wd.abs().t() * (dim * ULP / tau)
    lse = torch.logsumexp(z, 1)
    d_lse = dz.max(1).values + 4 * ULP * z.abs().max(1).values + (vocab + 8) * ULP + 4 * ULP * lse.abs()
    rel_q = (3 * arg + k + 6) * ULP
    zq = torch.gather(z, 1, at.clamp_min(0))
    logq = torch.where(q > 0, q.clamp_min(1e-300).log(), 0.0)
    d_loss = (q * (d_lse + dz.max(1).values + 2 * rel_q)[:, None]).sum(1)
    d_loss += ((rel_q + (k + 8) * ULP)[:, None] * q * (logq.abs() + zq.abs() + lse.abs()[:, None])).sum(1)
    g = dloss.double().abs() * tau
    p = torch.exp(z - lse[:, None])
    soft = torch.zeros(x.shape[0], vocab + 1, dtype=torch.float64, device=x.device)
    soft.scatter_add_(1, torch.where(at < 0, vocab, at), q)
    soft = soft[:, :vocab]
    d_exp = dz + d_lse[:, None] + 4 * ULP * (z.abs() + lse.abs()[:, None]) + 8 * ULP
    dl = (p - soft).abs() * g[:, None]
    d_dl = g[:, None] * (p * torch.expm1(d_exp) + soft * (rel_q + 4 * ULP)[:, None])
    d_dl += (dl + d_dl) * (rounding + 4 * ULP) + (p * g[:, None]) * 4 * ULP + TINY[x.dtype]
    live = (at >= 0).any(1)
    dl, d_dl = dl * live[:, None], d_dl * live[:, None]
    rows = int(live.sum())
    d_dx = d_dl @ wd.abs() + vocab * ULP * ((dl + d_dl) @ wd.abs())
    d_dw = d_dl.t() @ xd.abs() + rows * ULP * ((dl + d_dl).t() @ xd.abs())
    return d_loss * tau * tau * live, d_lse * live, d_dx, d_dw


def check_losses(x, w, dloss, ids, teacher, tau, put, what):
    """All forms of a loss on these inputs (CPU tensors; put: onto the GPU)."""
    vocab = w.shape[0]
    if teacher is None:
        at, q = O.target_weights(ids, vocab)
        arg = torch.zeros(x.shape[0], dtype=torch.float64)
        fwd, both, back = M.classifier_loss, M.classifier_loss_grads, M.classifier_loss_backward
        rest, kw = (put(ids),), {}
    else:
        at, q = O.teacher_weights(teacher, ids, vocab, tau)
        t = torch.where(at >= 0, teacher.double(), nan)
        arg = torch.nan_to_num((t.nan_to_num(-inf).max(1).values - t.nan_to_num(inf).min(1).values) / tau, posinf=0,
                               neginf=0)
        fwd, both, back = M.distill_loss, M.distill_loss_grads, M.distill_loss_backward
        rest, kw = (put(teacher), put(ids)), {"temperature": tau}
    live = (at >= 0).any(1)
    gx, gw, gd = put(x), put(w), put(dloss)
    clean = torch.where(live[:, None], x.double(), 0.0).to(x.dtype)
    want_loss, want_lse = O.loss(clean, w, at, q, tau)
    half = HALF[x.dtype]
    for form in ("forward", "both", "backward"):
        poison((2, x.shape[0]), tuple(x.shape), tuple(w.shape))
        rounding = half * (1 + half) * (2 if form == "both" else 1)
        if x.dtype == B and x.shape[0] <= 128 and put is on_gpu:
            # what is left of it is rounded and added (half of half); before that, nine bits of a fraction
            rounding = half * half + 2.0 ** -10
        b_loss, b_lse, b_dx, b_dw = bounds_of(clean, w, dloss, at, q, arg, tau, rounding)
        if form == "backward":
            lse = want_lse.float()
            dx, dw = back(gd, gx, gw, *rest, put(lse), **kw)
            want = O.grads(dloss, clean, w, at, q, tau, lse)
        else:
            if form == "forward":
                loss, lse = fwd(gx, gw, *rest, **kw)
            else:
                loss, lse, dx, dw = both(gd, gx, gw, *rest, **kw)
                want = O.grads(dloss, clean, w, at, q, tau)
            assert loss.dtype == lse.dtype == F
            close(loss, want_loss, b_loss, f"{what}: {form} loss")
            close(lse, want_lse, b_lse, f"{what}: {form} lse")
        if form != "forward":
            assert dx.dtype == x.dtype and dw.dtype == w.dtype
            close(dx, want[0], b_dx + half * (want[0].abs() + b_dx) + TINY[x.dtype], f"{what}: {form} dx")
            close(dw, want[1], b_dw + half * (want[1].abs() + b_dw) + TINY[x.dtype], f"{what}: {form} dw")


def on_gpu(t):
    return t.cuda()


@pytest.mark.parametrize("dtype", [F, B], ids=str)
@pytest.mark.parametrize("tokens,vocab,dim", SIZES)
def test_classifier_loss(tokens, vocab, dim, dtype):
    x, w, dloss, ids, _ = inputs(tokens, vocab, dim, dtype, 0, tokens + vocab)
    check_losses(x, w, dloss, ids, None, 1.0, on_gpu, "aligned")
    check_losses(x, w, dloss, ids.int(), None, 1.0, guarded, "off alignment")


@pytest.mark.parametrize("k,tau", [(1, 1.0), (5, 2.0), (64, 0.7), (65, 1.0), (256, 3.0)])
@pytest.mark.parametrize("dtype", [F, B], ids=str)
@pytest.mark.parametrize("tokens,vocab,dim", [(1, 16, 16), (5, 33, 7), (40, 2050, 264), (130, 300, 72), (257, 515, 129),
                                              (64, 5000, 40), (100, 700, 72), (700, 1000, 72), (300, 2050, 136)])
def test_distill_loss(tokens, vocab, dim, dtype, k, tau):
    x, w, dloss, ids, teacher = inputs(tokens, vocab, dim, dtype, k, tokens + k)
    check_losses(x, w, dloss, ids, teacher, tau, on_gpu, "aligned")
    check_losses(x, w, dloss, ids.int(), teacher.bfloat16(), tau, guarded, "off alignment")


@pytest.mark.parametrize("dtype", [F, B], ids=str)
@pytest.mark.parametrize("tokens", [1023, 8193, 16384, 16385, 40007])
def test_many_rows(tokens, dtype):
    """Rows' places are counted by one block or by all of them, in their order either way."""
    x, w, dloss, ids, _ = inputs(tokens, 40, 8, dtype, 0, tokens, absent=0.5)
    check_losses(x, w, dloss, ids, None, 1.0, on_gpu, "targets")
    x, w, dloss, ids, teacher = inputs(tokens, 40, 8, dtype, 3, tokens + 1, absent=0.5)
    check_losses(x, w, dloss, ids.int(), teacher, 1.5, on_gpu, "teacher")


@pytest.mark.parametrize("tokens,vocab", [(70, 150), (600, 1000), (60, 5000)])
def test_rows_that_do_not_count_are_not_read(tokens, vocab):
    """NaN and infinities in rows without a target reach nothing, in dw neither."""
    x, w, dloss, ids, _ = inputs(tokens, vocab, 48, F, 0, 3)
    ids[:5] = torch.tensor([3, -1, vocab, 7, -1])
    dead = O.named(ids, vocab) < 0
    x[dead] = torch.tensor([nan, inf, -inf])[torch.arange(int(dead.sum())) % 3][:, None]
    dloss[dead] = nan
    for dtype in (F, B):
        check_losses(x.to(dtype), w.to(dtype), torch.where(dead, 0.0, dloss), ids, None, 1.0, on_gpu, "dead rows")
        got = M.classifier_loss_grads(dloss.cuda(), x.to(dtype).cuda(), w.to(dtype).cuda(), ids.cuda())
        assert all(bool(t.isfinite().all()) for t in got)


@pytest.mark.parametrize("tokens,vocab", [(40, 90), (700, 1000), (40, 5000)])
def test_no_row_counts(tokens, vocab):
    for dtype in (F, B):
        x, w, dloss, ids, teacher = inputs(tokens, vocab, 24, dtype, 4, 8)
        none = torch.full((tokens,), -1).cuda()
        x, w, dloss, ids, teacher = (t.cuda() for t in (x, w, dloss, ids, teacher))
        for got in (M.classifier_loss_grads(dloss, x, w, none),
                    M.classifier_loss(x, w, none),
                    M.classifier_loss_backward(dloss, x, w, none, dloss),
                    M.distill_loss_grads(dloss, x, w, torch.full_like(teacher, -inf), ids),
                    M.distill_loss(x, w, teacher * nan, ids),
                    M.distill_loss_backward(dloss, x, w, teacher, ids * 0 - 5, dloss)):
            assert all(not t.any() for t in got)


def test_no_rows():
    for dtype in (F, B):
        x, w = torch.empty(0, 24, dtype=dtype).cuda(), torch.randn(90, 24).to(dtype).cuda()
        none, d = torch.empty(0, dtype=J).cuda(), torch.empty(0).cuda()
        poison((90, 24))
        loss, lse, dx, dw = M.classifier_loss_grads(d, x, w, none)
        assert loss.shape == lse.shape == (0,) and dx.shape == (0, 24) and not dw.any()
        assert not M.classifier_loss_backward(d, x, w, none, d)[1].any()
        t = torch.empty(0, 3).cuda()
        assert not M.distill_loss_grads(d, x, w, t, none.view(0, 1).expand(0, 3).contiguous())[3].any()
        assert M.classifier_loss(x, w, none)[0].shape == (0,)
        assert not M.embed_backward(x, none, 90).any() and M.embed(none, w).shape == (0, 24)


@pytest.mark.parametrize("tokens,vocab", [(60, 100), (700, 1000), (60, 5000)])
def test_teacher_entries_that_are_not_there(tokens, vocab):
    """-inf, NaN, +inf and ids of nothing in a teacher's rows, ids that come twice."""
    x, w, dloss, ids, teacher = inputs(tokens, vocab, 32, F, 6, 11)
    teacher[0, :3] = torch.tensor([-inf, nan, -inf])
    teacher[1] = -inf
    teacher[2, 1] = 3e38
    teacher[3, :] = -3e38
    teacher[4, 0] = -3.4e38
    ids[5] = 7
    ids[6] = torch.tensor([4, 4, 9, 4, 9, -1])
    ids[7] = -1
    ids[8, 0] = vocab
    for i in (0, 2, 3, 4):
        ids[i] = torch.arange(6) + i
    # the differences of 6e38 over tau overflow to weight 0, as the definition's do
    at, q = O.teacher_weights(teacher, ids, vocab, 1.0)
    got = M.distill_loss_grads(dloss.cuda(), x.cuda(), w.cuda(), teacher.cuda(), ids.cuda())
    arg = torch.full((tokens,), 40.0, dtype=torch.float64)
    b = bounds_of(x, w, dloss, at, q, arg, 1.0, 2 * HALF[F])
    want = (*O.loss(x, w, at, q), *O.grads(dloss, x, w, at, q))
    for g, v, e, name in zip(got, want, b, ("loss", "lse", "dx", "dw")):
        close(g, v, e + HALF[F] * (v.abs() + e), name)
    teacher[2, 1] = inf     # counts as the largest fp32: all of the weight
    again = M.distill_loss_grads(dloss.cuda(), x.cuda(), w.cuda(), teacher.cuda(), ids.cuda())
    assert all(torch.equal(p, r) for p, r in zip(got, again))


def test_large_and_equal_logits():
    """Logits far beyond exp's range, and all equal: lse is exact there."""
    w = torch.full((512, 64), 1.0)
    x = torch.full((3, 64), 4.0)
    x[1], x[2] = -40.0, 0.0
    loss, lse = M.classifier_loss(x.cuda(), w.cuda(), torch.tensor([0, 511, 3]).cuda())
    want = torch.tensor([256.0, -2560.0, 0.0]).double() + math.log(512)
    close(lse, want, want.abs() * 8 * ULP + (512 + 8) * ULP, "lse")
    close(loss, torch.full((3,), math.log(512)).double(), want.abs() * 12 * ULP + (512 + 8) * ULP, "loss")


@pytest.mark.parametrize("dtype", [F, B], ids=str)
@pytest.mark.parametrize("tokens,vocab,dim", [(5, 1000, 64), (150, 700, 128), (150, 701, 65), (150, 4003, 128)])
def test_losses_near_zero(tokens, vocab, dim, dtype):
    """A loss is log(1 + sum over the others of exp(l_v - l_y)): the target's logit in its sum and the one taken off
    are the same number, whatever it was rounded by.  So the loss is off by the others' part of it, their differences
    to the target's off by 2 dz and two roundings of each, and by a few roundings at the size of 1."""
    g = gen(tokens + dim)
    w = (torch.randn(vocab, dim, generator=g) / math.sqrt(dim)).to(dtype)
    y = torch.randint(0, vocab, (tokens,), generator=g)
    x = (torch.randn(tokens, dim, generator=g) * 0.5 + torch.linspace(14, 40, tokens)[:, None] * w[y].float()).to(dtype)
    loss, _ = M.classifier_loss(x.cuda(), w.cuda(), y.cuda())
    both = M.classifier_loss_grads(torch.ones(tokens).cuda(), x.cuda(), w.cuda(), y.cuda())[0]
    z = x.double() @ w.double().t()
    others = torch.where(torch.arange(vocab) == y[:, None], -inf, z - z.gather(1, y[:, None]))
    want = torch.log1p(others.exp().sum(1))
    assert float(want.min()) < 1e-3
    dz = (x.double().abs() @ w.double().abs().t()).max(1).values * dim * ULP
    bound = want * 2 * (2 * dz + 8 * ULP * z.abs().max(1).values + (vocab + 8) * ULP) + 4 * ULP
    close(loss, want, bound, "loss")
    close(both, want, bound, "loss with gradients")


@pytest.mark.parametrize("form", ["both", "backward"])
def test_equal_dloss_is_not_rounded(form):
    """Averaged losses have one dloss, whose rounding to bf16 (here by 0.0036) would be in every
    gradient.  All logits are 0 and targets different: a target's entry of dl, dloss (2^-10 - 1),
    may be off by 2^-10, others, dloss 2^-10, by nothing; the result by half a step."""
    T, V, d, g = 300, 1024, 40, 1.0036 / 256
    x, w = torch.randn(T, d, generator=gen(1)).bfloat16(), torch.zeros(V, d).bfloat16()
    targets, dloss = torch.randperm(V, generator=gen(2))[:T], torch.full((T,), g)
    if form == "both":
        dw = M.classifier_loss_grads(dloss.cuda(), x.cuda(), w.cuda(), targets.cuda())[3]
    else:
        lse = torch.full((T,), math.log(V))
        dw = M.classifier_loss_backward(dloss.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse.cuda())[1]
    at, q = O.target_weights(targets, V)
    want = O.grads(dloss, x, w, at, q, 1.0)[1]
    own = torch.zeros(V, d, dtype=torch.float64).index_add_(0, targets, x.double().abs() * g)
    # sums of T products; exp(-lse) by a logarithm of half a step off
    slack = 2.0 ** -10 * own + (T + 16) * ULP * (own + x.double().abs().sum(0) * g / V)
    close(dw, want, slack + HALF[B] * (want.abs() + slack), "dw")


def test_overflow_of_a_logit_is_nan_in_its_row_alone():
    x, w, dloss, ids, _ = inputs(66, 140, 32, F, 0, 4, absent=0.0)
    x[7] = 3e38
    w[:, 0] = 2.0
    loss, lse = M.classifier_loss(x.cuda(), w.cuda(), ids.cuda())
    assert lse[7].isnan() or lse[7].isinf()
    keep = torch.arange(66) != 7
    assert bool(lse.cpu()[keep].isfinite().all() and loss.cpu()[keep].isfinite().all())


@pytest.mark.parametrize("dtype", [F, B], ids=str)
def test_chunks(dtype):
    """More rows than one chunk's gradients of the logits hold: the weight gradient's sums
    go on over the chunks."""
    vocab, dim, tokens = 131072, 16, (4096 if dtype == F else 8192) + 321
    x, w, dloss, ids, _ = inputs(tokens, vocab, dim, dtype, 0, 21, absent=0.05)
    x, w, dloss, ids = (t.cuda() for t in (x, w, dloss, ids))
    loss, lse, dx, dw = M.classifier_loss_grads(dloss, x, w, ids)
    back = M.classifier_loss_backward(dloss, x, w, ids, lse)
    at, q = O.target_weights(ids, vocab)
    arg = torch.zeros(tokens, dtype=torch.float64, device="cuda")
    want_loss, want_lse = O.loss(x, w, at, q)
    b_loss, b_lse, b_dx, b_dw = bounds_of(x, w, dloss, at, q, arg, 1.0, 2 * HALF[dtype] * (1 + HALF[dtype]))
    close(loss, want_loss, b_loss, "loss")
    close(lse, want_lse, b_lse, "lse")
    half = HALF[dtype]
    want = O.grads(dloss, x, w, at, q)
    for got in ((dx, dw), back):
        close(got[0], want[0], 2 * b_dx + half * (want[0].abs() + b_dx) + TINY[dtype], "dx")
        close(got[1], want[1], 2 * b_dw + half * (want[1].abs() + b_dw) + TINY[dtype], "dw")


@pytest.mark.parametrize("tokens,vocab", [(400, 700), (900, 2050), (60, 5000)])
@pytest.mark.parametrize("k", [0, 8])
def test_bits_repeat(k, tokens, vocab):
    x, w, dloss, ids, teacher = (None if t is None else t.cuda() for t in inputs(tokens, vocab, 192, B, k, 9))
    def call():
        return M.distill_loss_grads(dloss, x, w, teacher, ids) if k else M.classifier_loss_grads(dloss, x, w, ids)
    first = call()
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(first, call()))


# ---------------------------------------------------- streams, graphs, the whole

def model_step(tokens, targets, table, w, teacher, ids, dloss):
    """Embedding, both losses on the same rows, and back to the table."""
    x = M.embed(tokens, table, scale=2.0)
    loss, lse, dx, dw = M.classifier_loss_grads(dloss, x, w, targets)
    kd, klse, dx2, dw2 = M.distill_loss_grads(dloss, x, w, teacher, ids, temperature=2.0)
    again = M.classifier_loss_backward(dloss, x, w, targets, lse)
    return (loss, lse, kd, klse, dx, dx2, dw, dw2, *again, M.embed_backward(dx, tokens, table.shape[0], scale=2.0),
            M.classifier_loss(x, w, targets)[0])


def step_inputs(seed, dtype=B, n=300, vocab=500, dim=128, k=8):
    g = gen(seed)
    table = torch.randn(vocab, dim, generator=g).to(dtype).cuda()
    w = (torch.randn(vocab, dim, generator=g) / 8).to(dtype).cuda()
    ids = torch.randint(-2, vocab, (n, k), generator=g).cuda()
    return (torch.randint(0, vocab, (n,), generator=g).cuda(), torch.randint(-20, vocab, (n,), generator=g).cuda(), table,
            w, torch.randn(n, k, generator=g).cuda(), ids, torch.randn(n, generator=g).cuda())


STEPS = pytest.mark.parametrize("sizes", [(300, 500, 128), (400, 2100, 136), (20, 500, 64), (100, 5000, 72)])


@STEPS
def test_a_step_on_a_stream_of_its_own(sizes):
    args = step_inputs(1, B, *sizes)
    want = model_step(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = model_step(*args)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = M.embed(args[0], args[2], scale=2.0, stream=s)
    loss, _ = M.classifier_loss(x, args[3], args[1], stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(loss, want[0])


@STEPS
@pytest.mark.parametrize("dtype", [F, B], ids=str)
def test_a_step_in_a_graph(dtype, sizes):
    """Captured once, replayed on other values with eager work between."""
    args = step_inputs(2, dtype, *sizes)
    model_step(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = model_step(*args)
    for seed in (3, 4, 5):
        for a, b in zip(args, step_inputs(seed, dtype, *sizes)):
            a.copy_(b)
        want = model_step(*args)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@STEPS
def test_two_calls_at_once(sizes):
    """Calls on two streams have workspaces of their own."""
    a, b = step_inputs(6, B, *sizes), step_inputs(7, B, *sizes)
    want = model_step(*a), model_step(*b)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(3):
        for i, (s, args) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(s):
                got[i].append(model_step(*args))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(p, q) for r in got[i] for p, q in zip(r, want[i]))


def test_a_tensor_that_requires_grad_is_refused():
    tokens, targets, table, w, teacher, ids, dloss = step_inputs(8)
    x = M.embed(tokens, table)
    w.requires_grad_()
    with pytest.raises(ValueError, match="w requires grad"):
        M.classifier_loss(x, w, targets)
    with torch.no_grad():
        M.classifier_loss(x, w, targets)


# ------------------------------------------------------------------ entry points

def test_outputs_off_16_bytes():
    """The entry point writes dx and dw at any alignment of their type, and nothing beside them."""
    import ctypes
    from matrix_orthogonalizing_optimizer_muon_amd import _lib as L
    for tokens, vocab, dim in ((300, 520, 72), (70, 33, 8), (600, 1000, 72)):
        x, w, dloss, ids, _ = (None if t is None else t.cuda() for t in inputs(tokens, vocab, dim, B, 0, 31))
        want = M.classifier_loss_grads(dloss, x, w, ids)
        need = ctypes.c_uint64()
        assert L.lib().muon_classifier_loss_workspace(1, tokens, vocab, dim, 1, ctypes.byref(need)) == 0
        ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
        loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        dx, dw = (torch.full((t.numel() + 16,), 7.0, dtype=B, device="cuda") for t in (x, w))
        assert L.lib().muon_classifier_loss_grads(
            dloss.data_ptr(), x.data_ptr(), w.data_ptr(), ids.data_ptr(), 8, 1, tokens, vocab, dim, loss.data_ptr(),
            lse.data_ptr(), dx.data_ptr() + 2, dw.data_ptr() + 2, ws.data_ptr(), need.value,
            torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        for got, t in ((dx, want[2]), (dw, want[3])):
            assert torch.equal(got[1:1 + t.numel()].view(t.shape), t)
            assert bool((got[0] == 7).all() and (got[1 + t.numel():] == 7).all())
        assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("tokens,vocab", [(90, 200), (700, 1000)])
def test_given_lse_is_taken_as_it_is(tokens, vocab):
    """The backward pass goes by the lse that it is given, a shifted one too."""
    x, w, dloss, ids, _ = inputs(tokens, vocab, 40, F, 0, 41, absent=0.0)
    at, q = O.target_weights(ids, vocab)
    lse = O.loss(x, w, at, q)[1].float() + 0.25
    dx, dw = M.classifier_loss_backward(dloss.cuda(), x.cuda(), w.cuda(), ids.cuda(), lse.cuda())
    want = O.grads(dloss, x, w, at, q, 1.0, lse)
    b = bounds_of(x, w, dloss, at, q, torch.zeros(tokens, dtype=torch.float64), 1.0, HALF[F])
    close(dx, want[0], b[2] + HALF[F] * (want[0].abs() + b[2]), "dx")
    close(dw, want[1], b[3] + HALF[F] * (want[1].abs() + b[3]), "dw")


@pytest.mark.parametrize("dtype", [F, B], ids=str)
def test_gradients_against_differences(dtype):
    """The loss's own differences: moving x and w along a direction by h moves the loss by <gradient, direction> h, up
    to h^2 / 2 times the curvature along it and twice the loss's rounding over h."""
    x, w, dloss, ids, teacher = inputs(40, 120, 32, F, 3, 17, absent=0.1)
    x, w = x.to(dtype).float(), w.to(dtype).float()
    g = gen(18)
    vx, vw = torch.randn(x.shape, generator=g), torch.randn(w.shape, generator=g) / 32 ** 0.5
    dloss = dloss.abs()

    def total(a, b):
        loss, _ = M.distill_loss(a.cuda(), b.cuda(), teacher.cuda(), ids.cuda(), temperature=2.0)
        return float((loss.double().cpu() * dloss).sum())
    dx, dw = M.distill_loss_grads(dloss.cuda(), x.to(dtype).cuda(), w.to(dtype).cuda(), teacher.cuda(), ids.cuda(),
                                  temperature=2.0)[2:]
    slope = float((dx.cpu().double() * vx).sum() + (dw.cpu().double() * vw).sum())
    h = 2.0 ** -7
    got = (total(x + h * vx, w + h * vw) - total(x - h * vx, w - h * vw)) / (2 * h)
    # third derivatives along the direction: those of the same sum in 64 bits, by its own differences
    def exact(s):
        at, q = O.teacher_weights(teacher, ids, 120, 2.0)
        return float((O.loss((x + s * vx).double(), (w + s * vw).double(), at, q, 2.0)[0] * dloss).sum())
    third = abs(exact(2 * h) - 2 * exact(h) + 2 * exact(-h) - exact(-2 * h)) / (2 * h ** 3)
    size = float((dx.cpu().double() * vx).abs().sum() + (dw.cpu().double() * vw).abs().sum())
    rounding = float(dloss.sum()) * 64 * 32 * ULP / h      # of 32-term logits of size 64 at the most
    assert abs(got - slope) <= third * h * h + rounding + 3 * HALF[dtype] * size, (got, slope)


@pytest.mark.parametrize("teacher", [False, True])
def test_example_runs_and_its_gradients_are_the_losses(teacher):
    """The model's gradients against differences of its loss along each tensor's gradient: the loss is piecewise smooth
    in the classifier, the last tensor of the chain, and in the table, the first."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "language_model.py")
    spec = importlib.util.spec_from_file_location("language_model", path)
    lm = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(lm)
    losses, model = lm.train(steps=3, vocab=500, tokens=256, width=64, hidden=64, experts=4)
    assert all(math.isfinite(v) for v in losses)
    if teacher:
        losses, model = lm.train(steps=3, vocab=500, tokens=256, width=64, hidden=64, experts=4, teacher=model, seed=3)
        assert all(math.isfinite(v) for v in losses)
    t, y = lm.text(500, 256, 3)
    top = model.top(t, 16) if teacher else None
    if top is not None:    # another distribution than the model's own, whose gradient is none
        top = (top[0].roll(1, dims=1).contiguous(), top[1])
    _, grads = model.loss_and_grads(t, y, top)
    for tensor, grad in ((model.classifier, grads[0]), (model.table, grads[1])):
        keep = tensor.clone()
        # steps of whole bf16 roundings are lost in weights of size 1/8, so a step is taken of the size of the weights
        way = grad.float() / grad.float().norm() * keep.float().norm() * 0.05
        sides = []
        for s in (1, -1):
            tensor.copy_((keep.float() + s * way).to(B))
            sides.append((float(model.loss_and_grads(t, y, top)[0]), tensor.float() - keep.float()))
            tensor.copy_(keep)
        moved = float(((sides[0][1] - sides[1][1]) * grad.float()).sum())
        assert moved > 0 and sides[0][0] > sides[1][0]
        # half a bf16 step in each of the layer's tensors, and the curvature over a step of a twentieth
        assert abs((sides[0][0] - sides[1][0]) / moved - 1) < 0.15
