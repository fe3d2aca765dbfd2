"""A gate for no rows, or for fewer, is refused, as gs_norm_gate_fwd refuses it."""

import pytest
import torch

from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("per", [0, -1, -7])
def test_rows_per_gate_below_one(per):
    x = torch.ones(7, 16, device="cuda")
    gate, stats = torch.ones(7, 16, device="cuda"), torch.ones(2, 7, device="cuda")
    for g in (gate, None):
        with pytest.raises(ValueError, match="rows_per_gate"):
            T.norm_gate(x, x, g, rows_per_gate=per)
        with pytest.raises(ValueError, match="rows_per_gate"):
            T.norm_gate_backward(x, x, x, x, g, None, None, stats, rows_per_gate=per)
    empty = torch.ones(0, 16, device="cuda")
    assert T.norm_gate(empty, empty)[0].shape == (0, 16)  # of no rows, one gate would hold none
