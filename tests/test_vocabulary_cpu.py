"""The vocabulary operators on the CPU: what the binding and the C entry points
refuse, calls with nothing to do, and the oracle's gradients against
differences.  Nothing here reaches a kernel."""
import ctypes
import math

import pytest
import torch

import matrix_orthogonalizing_optimizer_muon_amd as M
from matrix_orthogonalizing_optimizer_muon_amd import _lib as L
from oracle import vocabulary_oracle as O

F, B, I, J = torch.float32, torch.bfloat16, torch.int32, torch.int64


def z(*shape, dtype=F):
    return torch.zeros(shape, dtype=dtype)


X, W, T, D = z(4, 8), z(6, 8), z(4, dtype=J), z(4)
IDS, TEACHER = z(4, 3, dtype=J), z(4, 3)

REFUSALS = [
    (TypeError, "tokens is not a tensor", lambda: M.embed([1, 2], W)),
    (ValueError, "tokens must have 1 dimension, not 2", lambda: M.embed(z(2, 2, dtype=J), W)),
    (ValueError, "int32 or int64", lambda: M.embed(z(4), W)),
    (ValueError, "int32 or int64", lambda: M.embed(z(4, dtype=torch.int16), W)),
    (ValueError, "float32 or bfloat16", lambda: M.embed(T, z(6, 8, dtype=torch.float16))),
    (ValueError, "table must have 2", lambda: M.embed(T, z(8))),
    (ValueError, "not on the GPU", lambda: M.embed(T, W)),
    (ValueError, "dout has 4 rows for 5 tokens", lambda: M.embed_backward(X, z(5, dtype=J), 6)),
    (ValueError, "vocab must be >= 1", lambda: M.embed_backward(X, T, 0)),
    (ValueError, "not on the GPU", lambda: M.embed_backward(X, T, 6)),
    (ValueError, "x is torch.float32, w torch.bfloat16", lambda: M.classifier_loss(X, z(6, 8, dtype=B), T)),
    (ValueError, "x has 8 columns, w 7", lambda: M.classifier_loss(X, z(6, 7), T)),
    (ValueError, "targets has 5 rows, x 4", lambda: M.classifier_loss(X, W, z(5, dtype=J))),
    (ValueError, "targets must have 1 dimension", lambda: M.classifier_loss(X, W, IDS)),
    (ValueError, "targets must be int32 or int64", lambda: M.classifier_loss(X, W, D)),
    (ValueError, "not on the GPU", lambda: M.classifier_loss(X, W, T)),
    (ValueError, "dloss must be", lambda: M.classifier_loss_grads(z(4, dtype=B), X, W, T)),
    (ValueError, "dloss must be", lambda: M.classifier_loss_grads(z(3), X, W, T)),
    (ValueError, "lse must be", lambda: M.classifier_loss_backward(D, X, W, T, z(5))),
    (TypeError, "lse is not a tensor", lambda: M.classifier_loss_backward(D, X, W, T, None)),
    (ValueError, "not on the GPU", lambda: M.classifier_loss_backward(D, X, W, T, D)),
    (ValueError, "ids must have 2 dimensions", lambda: M.distill_loss(X, W, TEACHER, T)),
    (ValueError, r"teacher has shape \(4, 2\), ids \(4, 3\)", lambda: M.distill_loss(X, W, z(4, 2), IDS)),
    (ValueError, "teacher must be float32 or bfloat16", lambda: M.distill_loss(X, W, TEACHER.double(), IDS)),
    (ValueError, "temperature", lambda: M.distill_loss(X, W, TEACHER, IDS, temperature=0.0)),
    (ValueError, "temperature", lambda: M.distill_loss(X, W, TEACHER, IDS, temperature=-1.0)),
    (ValueError, "temperature", lambda: M.distill_loss(X, W, TEACHER, IDS, temperature=math.nan)),
    (ValueError, "temperature", lambda: M.distill_loss(X, W, TEACHER, IDS, temperature=math.inf)),
    (ValueError, "not on the GPU", lambda: M.distill_loss(X, W, TEACHER, IDS)),
    (ValueError, "dloss must be", lambda: M.distill_loss_grads(z(4, 1), X, W, TEACHER, IDS)),
    (ValueError, "lse must be", lambda: M.distill_loss_backward(D, X, W, TEACHER, IDS, D.double())),
]


@pytest.mark.parametrize("i", range(len(REFUSALS)))
def test_binding_refuses(i):
    kind, match, call = REFUSALS[i]
    with pytest.raises(kind, match=match):
        call()


# a non-NULL address that no refused call may touch
P, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4097)
N = None
BIG = 1 << 40


@pytest.mark.parametrize("want,name,args", [
    (L.MUON_EUNSUPPORTED, "muon_embed", (P, 2, P, 1, 4, 6, 8, 1.0, P, N)),
    (L.MUON_EUNSUPPORTED, "muon_embed", (P, 8, P, 2, 4, 6, 8, 1.0, P, N)),
    (L.MUON_EINVAL, "muon_embed", (P, 8, P, 1, -4, 6, 8, 1.0, P, N)),
    (L.MUON_EINVAL, "muon_embed", (P, 8, P, 1, 4, 0, 8, 1.0, P, N)),
    (L.MUON_EINVAL, "muon_embed", (P, 8, P, 1, 4, 6, 0, 1.0, P, N)),
    (L.MUON_EINVAL, "muon_embed", (N, 8, P, 1, 4, 6, 8, 1.0, P, N)),
    (L.MUON_EUNSUPPORTED, "muon_embed", (P, 8, P, 1, 1 << 31, 6, 8, 1.0, P, N)),
    (L.MUON_EUNSUPPORTED, "muon_embed", (P, 8, P, 1, 4, 1 << 31, 8, 1.0, P, N)),
    (L.MUON_EUNSUPPORTED, "muon_embed", (P, 8, P, 1, 4, 6, 1 << 24, 1.0, P, N)),
    (L.MUON_EINVAL, "muon_embed_backward", (P, P, 8, 1, 4, 6, 8, 1.0, P, N, 0, N)),
    (L.MUON_EINVAL, "muon_embed_backward", (P, P, 8, 1, 4, 6, 8, 1.0, P, P, 16, N)),
    (L.MUON_EINVAL, "muon_embed_backward", (P, P, 8, 1, 4, 6, 8, 1.0, P, ODD, BIG, N)),
    (L.MUON_EINVAL, "muon_embed_backward", (N, P, 8, 1, 4, 6, 8, 1.0, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_embed_backward", (N, N, 8, 1, 0, 6, 8, 1.0, N, P, BIG, N)),
    (L.MUON_EINVAL, "muon_embed_backward_workspace", (4, 6, 8, N)),
    (L.MUON_EINVAL, "muon_classifier_loss_workspace", (1, 4, 6, 8, 0, N)),
    (L.MUON_EINVAL, "muon_classifier_loss", (P, P, P, 8, 1, 4, 6, 8, P, N, P, BIG, N)),
    (L.MUON_EINVAL, "muon_classifier_loss", (P, P, N, 8, 1, 4, 6, 8, P, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_classifier_loss", (P, P, P, 8, 1, 4, 6, 8, P, P, N, 0, N)),
    (L.MUON_EINVAL, "muon_classifier_loss", (P, P, P, 8, 1, 4, 6, 8, P, P, P, 64, N)),
    (L.MUON_EINVAL, "muon_classifier_loss", (P, P, P, 8, 1, 4, 6, 8, P, P, ODD, BIG, N)),
    (L.MUON_EUNSUPPORTED, "muon_classifier_loss", (P, P, P, 1, 1, 4, 6, 8, P, P, P, BIG, N)),
    (L.MUON_EUNSUPPORTED, "muon_classifier_loss", (P, P, P, 8, 5, 4, 6, 8, P, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_classifier_loss_grads", (N, P, P, P, 8, 1, 4, 6, 8, P, P, P, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_classifier_loss_grads", (P, P, P, P, 8, 1, 4, 6, 8, P, N, P, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_classifier_loss_grads", (P, P, P, P, 8, 1, 4, 6, 8, P, P, N, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_classifier_loss_grads", (N, N, N, N, 8, 1, 0, 6, 8, N, N, N, N, P, BIG, N)),
    (L.MUON_EINVAL, "muon_classifier_loss_backward", (P, P, P, P, N, 8, 1, 4, 6, 8, P, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_classifier_loss_backward", (P, P, P, P, P, 8, 1, 4, 6, 8, P, N, P, BIG, N)),
    (L.MUON_EINVAL, "muon_distill_loss_workspace", (1, 4, 6, 8, 0, 0, ctypes.byref(ctypes.c_uint64()))),
    (L.MUON_EINVAL, "muon_distill_loss_workspace", (1, 4, 6, 8, 3, 3, ctypes.byref(ctypes.c_uint64()))),
    (L.MUON_EUNSUPPORTED, "muon_distill_loss_workspace", (1, 4, 6, 8, 257, 0, ctypes.byref(ctypes.c_uint64()))),
    (L.MUON_EUNSUPPORTED, "muon_distill_loss_workspace", (1, 1 << 24, 6, 8, 128, 0, ctypes.byref(ctypes.c_uint64()))),
    (L.MUON_EINVAL, "muon_distill_loss", (P, P, P, 0, P, 8, 1, 4, 6, 8, 0, 1.0, P, P, P, BIG, N)),
    (L.MUON_EUNSUPPORTED, "muon_distill_loss", (P, P, P, 0, P, 8, 1, 4, 6, 8, 257, 1.0, P, P, P, BIG, N)),
    (L.MUON_EUNSUPPORTED, "muon_distill_loss", (P, P, P, 3, P, 8, 1, 4, 6, 8, 3, 1.0, P, P, P, BIG, N)),
    (L.MUON_EUNSUPPORTED, "muon_distill_loss", (P, P, P, -1, P, 8, 1, 4, 6, 8, 3, 1.0, P, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_distill_loss", (P, P, P, 0, P, 8, 1, 4, 6, 8, 3, 0.0, P, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_distill_loss", (P, P, P, 0, P, 8, 1, 4, 6, 8, 3, math.nan, P, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_distill_loss", (P, P, N, 0, P, 8, 1, 4, 6, 8, 3, 1.0, P, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_distill_loss_grads", (P, P, P, P, 0, N, 8, 1, 4, 6, 8, 3, 1.0, P, P, P, P, P, BIG, N)),
    (L.MUON_EINVAL, "muon_distill_loss_backward", (P, P, P, P, 0, P, N, 8, 1, 4, 6, 8, 3, 1.0, P, P, P, BIG, N)),
])
def test_entry_point_refuses(want, name, args):
    lib = L.lib()
    assert getattr(lib, name)(*args) == want
    assert lib.muon_last_error()


def test_nothing_to_do():
    lib = L.lib()
    assert lib.muon_embed(N, 8, N, 1, 0, 6, 8, 1.0, N, N) == L.MUON_OK
    assert lib.muon_classifier_loss(N, N, N, 8, 1, 0, 6, 8, N, N, N, 0, N) == L.MUON_OK
    assert lib.muon_distill_loss(N, N, N, 0, N, 8, 1, 0, 6, 8, 3, 1.0, N, N, N, 0, N) == L.MUON_OK


def test_workspaces():
    """Workspaces grow with what a call keeps, and stay bounded where rows or vocabulary do not."""
    need = ctypes.c_uint64()

    def bytes_of(name, *args):
        assert getattr(L.lib(), name)(*args, ctypes.byref(need)) == L.MUON_OK
        return need.value
    tokens, vocab, dim = 4096, 32000, 1024
    loss, grads, given = (bytes_of("muon_classifier_loss_workspace", 1, tokens, vocab, dim, g) for g in (0, 1, 2))
    assert loss < tokens * vocab          # far from the logits' 2 or 4 bytes each
    assert loss < given <= grads
    # a million rows: dl within 2 GiB, the slabs' sums within 256 MiB, dw's sums, and what goes with
    # rows, a copy of x's live ones among it
    rows = (1 << 20) * (dim * 2 + 64)
    most = bytes_of("muon_classifier_loss_workspace", 1, 1 << 20, 131072, dim, 1)
    assert most < (1 << 31) + (1 << 28) + 131072 * dim * 4 + rows
    assert bytes_of("muon_classifier_loss_workspace", 1, 1 << 20, 131072, dim, 0) < (1 << 28) + rows


# ---------------------------------------------------------------------- oracle

def _case(k, seed, tau):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(5, 6, generator=g, dtype=torch.float64)
    w = torch.randn(9, 6, generator=g, dtype=torch.float64)
    dloss = torch.randn(5, generator=g, dtype=torch.float64)
    if not k:
        return x, w, dloss, *O.target_weights(torch.tensor([3, -1, 8, 9, 0]), 9)
    ids = torch.randint(-1, 10, (5, k), generator=g)
    ids[1] = -1
    ids[2, :2] = 4
    return x, w, dloss, *O.teacher_weights(torch.randn(5, k, generator=g), ids, 9, tau)


@pytest.mark.parametrize("k,tau", [(0, 1.0), (1, 1.0), (4, 2.0), (4, 0.5)])
def test_oracle_gradients_against_differences(k, tau):
    x, w, dloss, at, q = _case(k, 3 + k, tau)
    dx, dw = O.grads(dloss, x, w, at, q, tau)
    h = 1e-5
    for t, d in ((x, dx), (w, dw)):
        for i in range(t.numel()):
            keep = t.view(-1)[i].item()
            side = []
            for s in (h, -h):
                t.view(-1)[i] = keep + s
                side.append(float((O.loss(x, w, at, q, tau)[0] * dloss).sum()))
            t.view(-1)[i] = keep
            # central differences: h^2 times a third derivative of order 10, and 1e-16 / h of rounding
            assert abs((side[0] - side[1]) / (2 * h) - float(d.view(-1)[i])) < 1e-7


def test_oracle_loss_is_cross_entropy_and_divergence():
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(7, 4, generator=g).double(), torch.randn(11, 4, generator=g).double()
    targets = torch.tensor([0, 10, 3, -1, 5, 5, 11])
    loss, lse = O.loss(x, w, *O.target_weights(targets, 11))
    want = torch.nn.functional.cross_entropy(x @ w.t(), torch.where((targets < 0) | (targets > 10), -100, targets),
                                             reduction="none")
    assert torch.allclose(loss, want, rtol=1e-12, atol=1e-12)
    teacher = torch.randn(7, 11, generator=g).double()
    ids = torch.arange(11).expand(7, 11)
    at, q = O.teacher_weights(teacher, ids, 11, 2.0)
    loss, _ = O.loss(x, w, at, q, 2.0)
    want = 4 * torch.nn.functional.kl_div(torch.log_softmax(x @ w.t() / 2, 1), torch.softmax(teacher / 2, 1),
                                          reduction="none").sum(1)
    assert torch.allclose(loss, want, rtol=1e-12, atol=1e-12)


def test_oracle_embedding_gradient_is_the_adjoint():
    g = torch.Generator().manual_seed(2)
    table, dout = torch.randn(6, 3, generator=g).double(), torch.randn(9, 3, generator=g).double()
    t = torch.tensor([0, 5, 5, -1, 2, 6, 2, 2, 0])
    left = (O.embed(t, table, 3.0) * dout).sum()
    assert torch.allclose(left, (O.embed_backward(dout, t, 6, 3.0) * table).sum())
