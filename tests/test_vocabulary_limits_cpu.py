"""What the vocabulary operators refuse at the borders of their arguments.  Nothing
here reaches a kernel."""
import ctypes

import pytest
import torch

import matrix_orthogonalizing_optimizer_muon_amd as M
from matrix_orthogonalizing_optimizer_muon_amd import _lib as L

# a non-NULL address that no refused call may touch
P, N = ctypes.c_void_p(4096), None


@pytest.mark.parametrize("tau", [1e-45, 1e-39, 2.0 ** -64, 2.0 ** 64, 3e38])
def test_temperatures_whose_square_or_inverse_leaves_fp32(tau):
    """Such calls gave losses of 0, infinity or fewer digits for rows that count.  The workspace of none is refused last."""
    for call in ((lambda t: L.lib().muon_distill_loss(P, P, P, 0, P, 8, 1, 4, 6, 8, 3, t, P, P, N, 0, N)),
                 (lambda t: L.lib().muon_distill_loss_grads(P, P, P, P, 0, P, 8, 1, 4, 6, 8, 3, t, P, P, P, P, N, 0, N)),
                 (lambda t: L.lib().muon_distill_loss_backward(P, P, P, P, 0, P, P, 8, 1, 4, 6, 8, 3, t, P, P, N, 0, N))):
        assert call(tau) == L.MUON_EUNSUPPORTED
        assert call(2.0 ** -63) == call(2.0 ** 63) == L.MUON_EINVAL
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    teacher, ids = torch.zeros(4, 3), torch.zeros(4, 3, dtype=torch.int64)
    with pytest.raises(ValueError, match=r"temperature must be in \[2\^-63, 2\^63\]"):
        M.distill_loss(x, w, teacher, ids, temperature=tau)
    for ends in (2.0 ** -63, 2.0 ** 63):
        with pytest.raises(ValueError, match="not on the GPU"):
            M.distill_loss(x, w, teacher, ids, temperature=ends)
