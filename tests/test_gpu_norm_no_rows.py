"""The norms' gradients of no rows at all: the sums are written, as zeros."""

import pytest
import torch

from gaussian_splatting_differentiable_ewa_amd import _lib as L

pytestmark = pytest.mark.gpu


def test_sums_over_no_rows_are_zero():
    dev = "cuda"
    x, w, stats = torch.zeros(0, 40, device=dev), torch.ones(40, device=dev), torch.zeros(2, 0, device=dev)
    ws = torch.empty(L.norm_gate_bwd_workspace_bytes(0, 40, 4), dtype=torch.uint8, device=dev)
    gate = torch.ones(0, 40, device=dev)
    for f in (x, None):
        gw_post, gw_pre = torch.full((40,), 7.0, device=dev), torch.full((40,), 7.0, device=dev)
        L.gs_norm_gate_bwd(x, x, x, f, gate, w, w, stats, x, x, gate, gw_post, gw_pre, 4, ws)
        assert not gw_pre.any()
        assert not gw_post.any()
