"""The borders of the expert-layer entry points on the CPU: sizes of zero, sizes past
a limit, pointers that come in pairs.  Nothing here reaches a kernel."""
import ctypes

import pytest

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
