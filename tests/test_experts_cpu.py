"""The expert-layer operators on the CPU: what the binding and the C entry points
refuse, calls with nothing to do, and the oracle's gradients against
differences.  Nothing here reaches a kernel."""
import ctypes

import pytest
import torch

import matrix_orthogonalizing_optimizer_muon_amd as M
from matrix_orthogonalizing_optimizer_muon_amd import _lib as L
from oracle import experts_oracle as O

F, B, I = torch.float32, torch.bfloat16, torch.int32


def z(*shape, dtype=F):
    return torch.zeros(shape, dtype=dtype)


OFF = torch.tensor([0, 2, 4], dtype=I)

REFUSALS = [
    (TypeError, "logits is not a tensor", lambda: M.route([[1.0]], 1)),
    (ValueError, "float32 or bfloat16", lambda: M.route(z(4, 8, dtype=torch.float64), 2)),
    (ValueError, "2 dimensions", lambda: M.route(z(8), 2)),
    (ValueError, r"k must be in \[1, 8\]", lambda: M.route(z(4, 8), 9)),
    (ValueError, r"k must be in \[1, 8\]", lambda: M.route(z(4, 8), 0)),
    (ValueError, "not on the GPU", lambda: M.route(z(4, 8), 2)),
    (ValueError, "dweights must be", lambda: M.route_backward(
        z(4, 3), z(4, 8), M.Routing(z(4, 2), z(4, 2, dtype=I), z(4, 2, dtype=I), z(8, dtype=I), z(9, dtype=I)))),
    (ValueError, "experts must be", lambda: M.route_backward(
        z(4, 2), z(4, 8), M.Routing(z(4, 2), z(4, 2), z(4, 2, dtype=I), z(8, dtype=I), z(9, dtype=I)))),
    (ValueError, "x is torch.float32, w torch.bfloat16", lambda: M.grouped_matmul(z(4, 8), z(2, 3, 8, dtype=B), OFF)),
    (ValueError, "3 dimensions", lambda: M.grouped_matmul(z(4, 8), z(3, 8), OFF)),
    (ValueError, "x has 7 columns, w 8", lambda: M.grouped_matmul(z(4, 7), z(2, 3, 8), OFF)),
    (ValueError, "offsets has 3 entries for 5 experts", lambda: M.grouped_matmul(z(4, 8), z(5, 3, 8), OFF)),
    (ValueError, "offsets must be int32", lambda: M.grouped_matmul(z(4, 8), z(2, 3, 8), OFF.long())),
    (ValueError, "rows must be int32", lambda: M.grouped_matmul(z(4, 8), z(2, 3, 8), OFF, rows=z(4))),
    (ValueError, "not on the GPU", lambda: M.grouped_matmul(z(4, 8), z(2, 3, 8), OFF)),
    (ValueError, "dy has 8 columns, w 3 rows", lambda: M.grouped_input_grad(z(4, 8), z(2, 3, 8), OFF)),
    (ValueError, "not on the GPU", lambda: M.grouped_input_grad(z(4, 3), z(2, 3, 8), OFF)),
    (ValueError, "dy is torch.float32, x torch.bfloat16", lambda: M.grouped_weight_grad(z(4, 3), z(4, 8, dtype=B), OFF)),
    (ValueError, "dy has 4 rows, x or rows 5", lambda: M.grouped_weight_grad(z(4, 3), z(5, 8), OFF)),
    (ValueError, "dy has 4 rows, x or rows 6", lambda: M.grouped_weight_grad(z(4, 3), z(5, 8), OFF, rows=z(6, dtype=I))),
    (ValueError, "not on the GPU", lambda: M.grouped_weight_grad(z(4, 3), z(4, 8), OFF)),
    (ValueError, "y has 7 rows for 8 choices", lambda: M.combine(z(7, 8), z(4, 2, dtype=I), z(4, 2))),
    (ValueError, "weights must be", lambda: M.combine(z(8, 8), z(4, 2, dtype=I), z(4, 2, dtype=B))),
    (ValueError, "slots must be int32", lambda: M.combine(z(8, 8), z(4, 2), z(4, 2))),
    (ValueError, "dout must be", lambda: M.combine_backward(z(4, 7), z(8, 8), z(4, 2, dtype=I), z(4, 2), OFF)),
    (ValueError, "kind must be", lambda: M.checkpoint(z(4, 8), "int4")),
    (ValueError, "not on the GPU", lambda: M.checkpoint(z(4, 8), "int8")),
    (TypeError, "takes a Checkpoint", lambda: M.restore(z(4, 8))),
    (ValueError, "q must be int8", lambda: M.Checkpoint(z(4, 8), z(4, 1, dtype=torch.uint8), F)),
    (ValueError, "scale rows x ceil", lambda: M.Checkpoint(z(4, 33, dtype=torch.int8), z(4, 1, dtype=torch.uint8), F)),
    (ValueError, "unsupported dtype", lambda: M.Checkpoint(z(4, 8, dtype=torch.int8), z(4, 1, dtype=torch.uint8),
                                                           torch.float16)),
    (ValueError, "even number of columns", lambda: M.gated(z(4, 7))),
    (ValueError, "even number of columns", lambda: M.gated(z(4, 0))),
    (ValueError, "kind must be", lambda: M.gated(z(4, 8), checkpoint="fp8")),
    (ValueError, "gu must be", lambda: M.gated_backward(z(4, 8), z(4, 8))),
    (ValueError, "gu must be", lambda: M.gated_backward(z(4, 4, dtype=B), z(4, 8))),
    (ValueError, "not on the GPU", lambda: M.gated_backward(z(4, 4), z(4, 8))),
]


@pytest.mark.parametrize("i", range(len(REFUSALS)))
def test_binding_refuses(i):
    kind, match, call = REFUSALS[i]
    with pytest.raises(kind, match=match):
        call()


# a non-NULL address that no refused call may touch
P = ctypes.c_void_p(4096)
N = None


@pytest.mark.parametrize("want,name,args", [
    (L.MUON_EUNSUPPORTED, "muon_route", (P, 7, 4, 8, 2, 1, P, P, P, P, P, N, 0, N)),
    (L.MUON_EINVAL, "muon_route", (P, 0, -1, 8, 2, 1, P, P, P, P, P, N, 0, N)),
    (L.MUON_EINVAL, "muon_route", (P, 0, 4, 8, 9, 1, P, P, P, P, P, N, 0, N)),
    (L.MUON_EINVAL, "muon_route", (N, 0, 4, 8, 2, 1, P, P, P, P, P, N, 0, N)),
    (L.MUON_EINVAL, "muon_route", (N, 0, 0, 8, 2, 1, N, N, N, N, N, N, 0, N)),
    (L.MUON_EINVAL, "muon_route", (P, 0, 100000, 8, 2, 1, P, P, P, P, P, N, 0, N)),       # no workspace
    (L.MUON_EINVAL, "muon_route", (P, 0, 100000, 8, 2, 1, P, P, P, P, P, P, 8, N)),       # too small a one
    (L.MUON_EINVAL, "muon_route", (P, 0, 100000, 8, 2, 1, P, P, P, P, P, ctypes.c_void_p(4097), 1 << 40, N)),
    (L.MUON_EUNSUPPORTED, "muon_route", (P, 0, 4, 1025, 2, 1, P, P, P, P, P, N, 0, N)),
    (L.MUON_EUNSUPPORTED, "muon_route", (P, 0, 4, 128, 65, 1, P, P, P, P, P, N, 0, N)),
    (L.MUON_EUNSUPPORTED, "muon_route", (P, 0, 1 << 30, 8, 2, 1, P, P, P, P, P, N, 0, N)),
    (L.MUON_EINVAL, "muon_route_backward", (P, P, N, P, 0, 4, 8, 2, 1, P, N)),
    (L.MUON_EINVAL, "muon_route_workspace", (4, 8, N)),
    (L.MUON_EINVAL, "muon_grouped_matmul", (P, P, P, N, 1, 4, 5, 2, 8, 8, P, N)),          # x_rows != n
    (L.MUON_EINVAL, "muon_grouped_matmul", (P, P, N, P, 1, 4, 5, 2, 8, 8, P, N)),
    (L.MUON_EINVAL, "muon_grouped_matmul", (P, P, P, P, 1, -4, 5, 2, 8, 8, P, N)),
    (L.MUON_EINVAL, "muon_grouped_matmul", (P, P, P, P, 1, 4, 5, 0, 8, 8, P, N)),
    (L.MUON_EINVAL, "muon_grouped_matmul", (P, P, P, P, 1, 4, 5, 2, 8, 0, P, N)),
    (L.MUON_EUNSUPPORTED, "muon_grouped_matmul", (P, P, P, P, 2, 4, 5, 2, 8, 8, P, N)),
    (L.MUON_EUNSUPPORTED, "muon_grouped_matmul", (P, P, P, P, 1, 4, 5, 1025, 8, 8, P, N)),
    (L.MUON_EUNSUPPORTED, "muon_grouped_matmul", (P, P, P, P, 1, 1 << 31, 5, 2, 8, 8, P, N)),
    (L.MUON_EUNSUPPORTED, "muon_grouped_matmul", (P, P, P, P, 1, 4, 5, 2, 1 << 24, 8, P, N)),
    (L.MUON_EINVAL, "muon_grouped_input_grad", (P, P, P, 1, 4, 2, 8, 8, N, N)),
    (L.MUON_EINVAL, "muon_grouped_weight_grad", (P, P, P, P, 0, P, N, 1, 4, 4, 2, 8, 8, P, P, 1 << 40, N)),   # x and q
    (L.MUON_EINVAL, "muon_grouped_weight_grad", (P, N, P, N, 0, P, N, 1, 4, 4, 2, 8, 8, P, P, 1 << 40, N)),   # no scale
    (L.MUON_EINVAL, "muon_grouped_weight_grad", (P, N, N, N, 0, P, N, 1, 4, 4, 2, 8, 8, P, P, 1 << 40, N)),   # no x
    (L.MUON_EUNSUPPORTED, "muon_grouped_weight_grad", (P, N, P, P, 5, P, N, 1, 4, 4, 2, 8, 8, P, P, 1 << 40, N)),
    (L.MUON_EINVAL, "muon_grouped_weight_grad_workspace", (1, 4, 4, 2, 8, 8, 1, N)),
    (L.MUON_EINVAL, "muon_combine", (P, P, P, 1, 4, 0, 8, P, N)),
    (L.MUON_EINVAL, "muon_combine", (P, P, P, 1, 4, 2, 0, P, N)),
    (L.MUON_EINVAL, "muon_combine", (P, N, P, 1, 4, 2, 8, P, N)),
    (L.MUON_EINVAL, "muon_combine_backward", (P, P, P, P, N, 1, 4, 2, 2, 8, P, P, N)),
    (L.MUON_EINVAL, "muon_checkpoint", (N, 1, 4, 8, 0, P, P, N)),
    (L.MUON_EUNSUPPORTED, "muon_checkpoint", (P, 1, 4, 8, 2, P, P, N)),
    (L.MUON_EUNSUPPORTED, "muon_checkpoint", (P, 1, 1 << 32, 8, 0, P, P, N)),
    (L.MUON_EINVAL, "muon_restore", (P, N, 0, 4, 8, 1, P, N)),
    (L.MUON_EINVAL, "muon_gated", (P, 1, 4, 8, 0, P, P, N, N)),                            # q without scale
    (L.MUON_EINVAL, "muon_gated", (N, 1, 4, 8, 0, P, N, N, N)),
    (L.MUON_EINVAL, "muon_gated_backward", (P, P, P, P, 0, 1, 4, 8, P, P, N)),             # gu and q
    (L.MUON_EINVAL, "muon_gated_backward", (P, N, N, N, 0, 1, 4, 8, P, P, N)),
])
def test_entry_point_refuses(want, name, args):
    assert getattr(L.lib(), name)(*args) == want
    assert L.lib().muon_last_error()


def test_nothing_to_do_needs_no_device():
    lib = L.lib()
    assert lib.muon_grouped_matmul(N, P, P, P, 1, 0, 5, 2, 8, 8, N, N) == L.MUON_OK
    assert lib.muon_grouped_input_grad(N, P, P, 1, 0, 2, 8, 8, N, N) == L.MUON_OK
    assert lib.muon_combine(N, N, N, 1, 0, 2, 8, N, N) == L.MUON_OK
    assert lib.muon_combine_backward(N, N, N, N, N, 1, 0, 2, 2, 8, N, N, N) == L.MUON_OK
    assert lib.muon_checkpoint(N, 1, 0, 8, 0, N, N, N) == L.MUON_OK
    assert lib.muon_restore(N, N, 0, 0, 8, 1, N, N) == L.MUON_OK
    assert lib.muon_gated(N, 1, 0, 8, 0, N, N, N, N) == L.MUON_OK
    assert lib.muon_gated_backward(N, N, N, N, 0, 1, 0, 8, N, N, N) == L.MUON_OK
    assert lib.muon_route_backward(N, N, N, N, 0, 0, 8, 2, 1, N, N) == L.MUON_OK


def test_unknown_attribute():
    with pytest.raises(AttributeError):
        M.no_such_operator
    assert M.route is M.experts.route
    assert set(M.experts.__all__) <= set(M.__all__)


def test_checkpoint_describes_itself():
    c = M.Checkpoint(z(4, 33, dtype=torch.int8), z(4, 2, dtype=torch.uint8), B)
    assert tuple(c.shape) == (4, 33) and c.nbytes == 4 * 33 + 8 and c.dtype == B


def _difference(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("normalize", [True, False])
def test_oracle_router_gradient_against_differences(normalize):
    g = torch.Generator().manual_seed(3)
    l = torch.randn(6, 9, generator=g, dtype=torch.float64)
    l[2, 4] = -float("inf")
    l[3] = -float("inf")
    dw = torch.randn(6, 3, generator=g, dtype=torch.float64)
    d = torch.randn(6, 9, generator=g, dtype=torch.float64)
    got = (O.route_backward(dw, l, 3, normalize) * d).sum()
    want = _difference(lambda x: (O.route(x, 3, normalize)[0] * dw).sum(), l, d)
    # central differences: h^2 times third derivatives of O(1), and 1e-16 / h of rounding
    assert abs(got - want) < 1e-8


def test_oracle_layer_gradients_against_differences():
    g = torch.Generator().manual_seed(4)

    def r(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)
    l = r(7, 4)
    _, _, slots, rows, off = O.route(l, 2)
    slots, rows = torch.tensor(slots), torch.tensor(rows)
    x, w, gu, dy, wt = r(7, 5), r(4, 6, 5), r(14, 8), r(14, 6), r(7, 2)
    dx, dw_, dgu, dd = r(14, 5), r(4, 6, 5), r(14, 8), r(14, 4)
    v = O.gathered(x, rows)
    assert abs((O.input_grad(dy, w, off) * dx).sum() -
               _difference(lambda t: (O.matmul(t, w, off) * dy).sum(), v, dx)) < 1e-7
    assert abs((O.weight_grad(dy, x, off, rows) * dw_).sum() -
               _difference(lambda t: (O.matmul(x, t, off, rows) * dy).sum(), w, dw_)) < 1e-7
    assert abs((O.gated_backward(dd, gu) * dgu).sum() -
               _difference(lambda t: (O.gated(t) * dd).sum(), gu, dgu)) < 1e-7
    y, dout, ey, ew = r(14, 3), r(7, 3), r(14, 3), r(7, 2)
    a, b = O.combine_backward(dout, y, slots, wt)
    assert abs((a * ey).sum() - _difference(lambda t: (O.combine(t, slots, wt) * dout).sum(), y, ey)) < 1e-7
    assert abs((b * ew).sum() - _difference(lambda t: (O.combine(y, slots, t) * dout).sum(), wt, ew)) < 1e-7


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_oracle_checkpoint_error_is_half_a_step(kind):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(4, 70, generator=g, dtype=torch.float64) * torch.exp(3 * torch.randn(4, 1, generator=g,
                                                                                         dtype=torch.float64))
    q, scale, back = O.checkpoint(x, kind)
    s = torch.pow(2.0, scale.double() - 127).repeat_interleave(32, 1)[:, :70]
    step = s if kind == "int8" else torch.maximum(back.abs() * 2.0 ** -3, s * 2.0 ** -9)
    # int8: a value that rounds to 128 steps is held as 127, so off by a whole one at most
    assert ((back - x).abs() <= step * (1.0 if kind == "int8" else 0.5) * (1 + 1e-12)).all()
    assert q.abs().max() <= (127 if kind == "int8" else 448)
