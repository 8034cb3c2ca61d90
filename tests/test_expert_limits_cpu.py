"""The borders of the expert-layer entry points on the CPU: sizes of zero, sizes past
a limit, pointers that come in pairs.  Nothing here reaches a kernel."""
import contextlib
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import matrix_orthogonalizing_optimizer_muon_amd as M
from matrix_orthogonalizing_optimizer_muon_amd import _lib as L

# a non-NULL address that no refused call may touch
P = ctypes.c_void_p(4096)
N = None


@pytest.mark.parametrize("n", [0, 4])
@pytest.mark.parametrize("q,scale", [(P, N), (N, P)])
def test_weight_grad_takes_no_half_checkpoint(n, q, scale):
    """Also with no rows to sum over, where the checkpoint would not be needed."""
    rc = L.lib().muon_grouped_weight_grad(P, N, q, scale, L.MUON_INT8, P, P, L.MUON_BF16, n, 4, 2, 8, 8, P, P, 1 << 40, N)
    assert rc == L.MUON_EINVAL


def test_weight_grad_of_no_rows_needs_no_workspace():
    for kept in (0, 1):
        need = ctypes.c_uint64(99)
        assert L.lib().muon_grouped_weight_grad_workspace(L.MUON_BF16, 0, 4096, 2, 8, 8, kept, ctypes.byref(need)) == L.MUON_OK
        assert need.value == 0


NOTHING_OF_MANY_COLUMNS = """
import sys
sys.path.insert(0, {root!r})
import matrix_orthogonalizing_optimizer_muon_amd as M
from matrix_orthogonalizing_optimizer_muon_amd import _lib as L
lib, N = L.lib(), None
for cols in (1 << 33, 1 << 35, (1 << 35) + 1, (1 << 62) + 8, (1 << 63) - 1):
    assert lib.muon_checkpoint(N, 1, 0, cols, 0, N, N, N) == L.MUON_OK, cols
    assert lib.muon_restore(N, N, 0, 0, cols, 1, N, N) == L.MUON_OK, cols
    assert lib.muon_gated(N, 1, 0, cols, 0, N, N, N, N) == L.MUON_OK, cols
    assert lib.muon_gated_backward(N, N, N, N, 0, 1, 0, cols, N, N, N) == L.MUON_OK, cols
    assert lib.muon_combine(N, N, N, 1, 0, 2, cols, N, N) == L.MUON_OK, cols
    assert lib.muon_combine_backward(N, N, N, N, N, 1, 0, 2, 2, cols, N, N, N) == L.MUON_OK, cols
"""


def test_nothing_to_do_at_any_width():
    """Zero rows of so many columns that a count of column groups wraps to zero; in a process of its own, which a
    division by that count would end."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", NOTHING_OF_MANY_COLUMNS.format(root=root)], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr)


@pytest.mark.parametrize("cols", [(1 << 34) + 1, 1 << 35, (1 << 62) + 8, (1 << 63) - 1])
def test_more_columns_than_a_launch_has(cols):
    lib = L.lib()
    for rows in (1, 3):
        assert lib.muon_checkpoint(P, 1, rows, cols, 0, P, P, N) == L.MUON_EUNSUPPORTED
        assert lib.muon_restore(P, P, 0, rows, cols, 1, P, N) == L.MUON_EUNSUPPORTED
        assert lib.muon_gated(P, 1, rows, cols, 0, P, N, N, N) == L.MUON_EUNSUPPORTED
        assert lib.muon_gated(P, 1, rows, cols, 0, P, P, P, N) == L.MUON_EUNSUPPORTED
        assert lib.muon_gated_backward(P, P, N, N, 0, 1, rows, cols, P, P, N) == L.MUON_EUNSUPPORTED
        assert lib.muon_combine(P, P, P, 1, rows, 2, cols, P, N) == L.MUON_EUNSUPPORTED


# ----------------------------------------------------------- tensors that require grad

def g(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, requires_grad=True)


def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


OFF = torch.tensor([0, 2, 4], dtype=torch.int32)
SLOTS = torch.zeros(4, 2, dtype=torch.int32)
GRADS = {
    "route": ("logits", lambda: M.route(g(4, 8), 2)),
    "route_backward": ("logits", lambda: M.route_backward(z(4, 2), g(4, 8), M.Routing(z(4, 2), SLOTS, SLOTS, SLOTS, OFF))),
    "matmul, x": ("x", lambda: M.grouped_matmul(g(4, 8), z(2, 3, 8), OFF)),
    "matmul, w": ("w", lambda: M.grouped_matmul(z(4, 8), g(2, 3, 8), OFF, rows=OFF)),
    "input grad": ("w", lambda: M.grouped_input_grad(z(4, 3), g(2, 3, 8), OFF)),
    "weight grad": ("x", lambda: M.grouped_weight_grad(z(4, 3), g(4, 8), OFF)),
    "combine": ("weights", lambda: M.combine(z(8, 8), SLOTS, g(4, 2))),
    "combine_backward": ("y", lambda: M.combine_backward(z(4, 8), g(8, 8), SLOTS, z(4, 2), OFF)),
    "checkpoint": ("x", lambda: M.checkpoint(g(4, 8))),
    "gated": ("gu", lambda: M.gated(g(4, 8))),
    "gated_backward": ("gu", lambda: M.gated_backward(z(4, 4), g(4, 8))),
}


@pytest.mark.parametrize("name", list(GRADS))
def test_a_tensor_that_requires_grad_is_refused(name):
    """Its gradient would be lost: no call is recorded by autograd."""
    arg, call = GRADS[name]
    with pytest.raises(ValueError, match=f"{arg} requires grad"):
        call()
    with torch.no_grad(), pytest.raises(ValueError, match="is not on the GPU"):
        call()                                    # taken as far as where it lies


# ------------------------------------------------------------------------- streams

class OnGpu1(torch.Tensor):
    device = property(lambda self: torch.device("cuda:1"))


class OtherStream:
    device = torch.device("cuda:0")


def test_a_stream_is_of_the_tensors_gpu(monkeypatch):
    """A handle is taken as one of the tensors' GPU, whichever is current; a Stream of another GPU is refused."""
    from matrix_orthogonalizing_optimizer_muon_amd import experts as E
    seen = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda *a, **kw: seen.append((a, kw)) or "stream")
    monkeypatch.setattr(torch.cuda, "stream", lambda s: seen.append(s) or contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "Stream", OtherStream)
    x = z(4).as_subclass(OnGpu1)
    op = E._on(lambda x: "ran")
    assert op(x, stream=5) == op(x=x, stream=5) == "ran"
    assert seen == [((5,), {"device": torch.device("cuda:1")}), "stream"] * 2
    with pytest.raises(ValueError, match="stream is of cuda:0, the tensors are on cuda:1"):
        op(x, stream=OtherStream())


def test_tensors_off_the_gpu_are_refused_with_a_stream_too():
    with pytest.raises(ValueError, match="not on the GPU"):
        M.route(z(4, 8), 2, stream=0)
    with pytest.raises(TypeError, match="takes a Checkpoint"):
        M.restore([1], stream=0)


# ------------------------------------------------------------------------- router

@pytest.mark.parametrize("tokens,experts,scan", [
    (16384, 64, False), (32768, 64, False), (32769, 64, True), (65536, 64, True), (16384, 128, False),
    (16385, 128, True), (65, 129, True), (4096, 256, True), (65536, 256, True), (65536, 1024, True),
    (32768, 8, False), (32769, 8, True), (64, 1024, None)])
def test_route_scans_where_the_counts_are_many(tokens, experts, scan):
    """A placing block reads every block's counts of all experts where the scan does not: 32 KiB at most, of at most 128
    experts.  The workspace shows which (None: one block does it all and needs none)."""
    need = ctypes.c_uint64()
    assert L.lib().muon_route_workspace(tokens, experts, ctypes.byref(need)) == L.MUON_OK
    blocks = -(-tokens // 64)
    stride = -(-blocks // 16) * 16
    counts = -(-(blocks * 8 + stride) * experts // 16) * 16        # masks and counts
    assert need.value == (0 if scan is None else counts + (4 * (blocks + 1) * experts if scan else 0))


# ---------------------------------------------------------------- weight gradient

@pytest.mark.parametrize("dtype,n,experts,outer,inner,some", [
    (L.MUON_BF16, 100000, 128, 128, 128, False), (L.MUON_BF16, 100000, 128, 256, 128, False),
    (L.MUON_BF16, 100000, 128, 129, 128, True), (L.MUON_F32, 100000, 128, 64, 64, True),
    (L.MUON_BF16, 100000, 64, 128, 128, True), (L.MUON_BF16, 28945, 5, 64, 1280, True)])
def test_weight_grad_asks_for_no_workspace_that_it_leaves(dtype, n, experts, outer, inner, some):
    """The parts' sums, where the tiles that make them take the sizes."""
    need = ctypes.c_uint64(99)
    assert L.lib().muon_grouped_weight_grad_workspace(dtype, n, n, experts, outer, inner, 0, ctypes.byref(need)) == L.MUON_OK
    assert (need.value > 0) == some
