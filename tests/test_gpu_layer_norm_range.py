"""Layer norm of rows far above and below one: the sum of squared deviations has
to fit fp32, and does from 2^-60 to 2^55 at these lengths; with eps = 0
the result does not depend on a row's size."""

import pytest
import torch

import dense_oracle as O
from gaussian_splatting_differentiable_ewa_amd import tokens as T
from test_gpu_layer_norm import BF16, F32, gen, rand, rel

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [64, 1027, 2600])
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -30, 2.0 ** 30, 2.0 ** 55])
def test_both_ways(dtype, c, size):
    g = gen(c)
    x1, gy = (1.5 * rand(g, 40, c) + 0.8).to(dtype), rand(g, 40, c, dtype=dtype)
    w, b = 1 + 0.3 * rand(g, c), rand(g, c)
    x = x1 * size
    y, stats = T.layer_norm(x, w, b, 0.0)
    gx, gw, gb = T.layer_norm_backward(gy, x, w, stats)
    want = O.layer_norm(x1, w, b, 0.0)
    xd = x1.double()
    x0 = xd - xd.mean(-1, keepdim=True)
    mag = (x0.abs() + xd.abs().mean(-1, keepdim=True)) / (x0 ** 2).mean(-1, keepdim=True).sqrt() * w.double().abs() + b.double().abs()
    O.within(y, want, O.U[dtype] * want.abs() + 3 * rel(c) * mag + O.TINY[dtype], "y")
    (vx, mx), (vw, mw), (vb, mb) = O.layer_norm_gradients(gy, x1, w, 0.0)
    O.within(gx.double() * size, vx, O.U[dtype] * vx.abs() + 6 * rel(c) * mx + O.TINY[dtype] * size, "gx")
    chain = (40 + 64) * O.E
    O.within(gw, vw, (6 * rel(c) + chain) * mw, "gw")
    O.within(gb, vb, chain * mb, "gb")


def test_past_it():
    """A row whose squared deviations pass fp32 counts as infinitely wide; rows beside it are as without it."""
    g = gen(1)
    x, b = rand(g, 5, 96), rand(g, 96)
    y = T.layer_norm(x, None, b)[0]
    x[2] *= 2.0 ** 80
    y2, stats = T.layer_norm(x, None, b)
    rest = [0, 1, 3, 4]
    assert torch.equal(y2[rest], y[rest]) and torch.equal(y2[2], b) and stats[1, 2] == 0
