"""4-bit linear layers in tiles of 256 x 256 (taken from 192 of them on), whole
and ragged, against their definition in 64 bits."""

import math

import pytest
import torch

import dense_oracle as O
from gaussian_splatting_differentiable_ewa_amd import tokens as T
from test_gpu_fp4 import BF16, DEV, F16, F32, gen, rand

pytestmark = pytest.mark.gpu

# rows and columns whole and off the tiles, many of either; one block, a stage and less, and many stages
SIZES = [(4096, 512, 4096), (3300, 160, 4100), (6145, 32, 2049), (49153, 96, 255), (200, 416, 49200), (8200, 2080, 1800),
         (2049, 128, 6150)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,c,n", SIZES)
def test_linear(dtype, rows, c, n):
    assert -(-rows // 256) * -(-n // 256) >= 192
    g = gen(rows + c + n)
    x = rand(g, rows, c, dtype=dtype)
    weights = T.quantise4(rand(g, n, c) / math.sqrt(c))
    weights[1][:, c // 32:] = 255  # what fills a row up is not used
    got = T.linear4(x, weights)
    qx, qw = O.quantise4(x)[2], O.unpack4(*weights, c)
    want = qx @ qw.T
    mag = qx.abs() @ qw.abs().T
    O.within(got, want, O.U[dtype] * want.abs() + (c + 16) * O.E * mag + O.TINY[dtype], "y")
    assert torch.equal(T.linear4(x, weights), got)


def test_strides_and_what_is_not_finite():
    """Views with strides, rows off 16 bytes, scales of views; a NaN in a row reaches that row only, one in a weight
    that column only."""
    g = gen(3)
    rows, c, n = 3300, 160, 4100
    wide = rand(g, rows, 2 * c + 3, dtype=BF16)
    weights = T.quantise4(rand(g, n, 2 * c))
    part = weights[0][:, c // 2:], weights[1][:, 4:][:, :8]  # blocks from 4 on: not those of the codes, but valid
    same = part[0].contiguous(), part[1].contiguous()
    for first in (0, 3, c):
        x = wide[:, first: first + c]
        assert torch.equal(T.linear4(x, part), T.linear4(x.contiguous(), same))
    x = wide[:, :c].clone()
    y = T.linear4(x, same)
    x[3001, 70], same[1][2, 1] = float("nan"), 255
    y2 = T.linear4(x, same)
    bad = torch.zeros_like(y, dtype=torch.bool, device=DEV)
    bad[3001], bad[:, 2] = True, True
    assert torch.isnan(y2[bad]).all() and torch.equal(y2[~bad], y[~bad])
