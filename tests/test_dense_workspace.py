"""The gated feed-forward block's forward workspace: refused where it is missing,
off 16 bytes or short, before any HIP call (so without a GPU)."""

import ctypes

import pytest

from gaussian_splatting_differentiable_ewa_amd import _lib as L
from test_dense_abi import FAKE, INV, call, lib, mat  # noqa: F401  (lib: a fixture)


# sums in splits: of h and y, of h alone, of y alone
@pytest.mark.parametrize("rows,c,hidden,out", [(17, 2048, 8192, 2048), (17, 1008, 8, 128), (18, 8, 1456, 8)])
def test_forward_workspace_refusals(lib, rows, c, hidden, out):  # noqa: F811
    need = L.gated_ff_fwd_workspace_bytes(rows, c, hidden, out)
    assert need > 0
    w = mat(stride=8192)
    fwd = dict(x=w, wg=w, wu=w, wd=w, rows=rows, c=c, hid=hidden, co=out, act=L.GS_SILU, t=L.GS_BF16, h=FAKE, kept=FAKE, y=FAKE,
               ws=FAKE, wsb=need, s=None)
    for bad in (dict(ws=None), dict(ws=ctypes.c_void_p(4100)), dict(wsb=0), dict(wsb=need - 1)):
        assert call(lib.gs_gated_ff_fwd, fwd, **bad) == INV, bad
