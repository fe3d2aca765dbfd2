"""Layer norm, the gated feed-forward block and the 4-bit calls on matrices of
more than 2^31 elements: the last rows are those of the same call on them alone."""

import math

import pytest
import torch

import dense_oracle as O
from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

BF16, DEV = torch.bfloat16, "cuda"
LAST = 100


def rand(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=BF16)


def test_layer_norm():
    g = torch.Generator(device=DEV).manual_seed(1)
    rows, c = 140000, 16384
    x, w = torch.zeros(rows, c, dtype=BF16, device=DEV), 1 + torch.rand(c, generator=g, device=DEV)
    x[-LAST:] = rand(g, LAST, c)
    y, stats = T.layer_norm(x, w, None)
    few, fstats = T.layer_norm(x[-LAST:], w, None)
    assert torch.equal(y[-LAST:], few) and not y[:-LAST].any()
    gx, gw, _ = T.layer_norm_backward(y, x, w, stats)
    fgx, fgw, _ = T.layer_norm_backward(few, x[-LAST:], w, fstats)
    assert torch.equal(gx[-LAST:], fgx)
    # both sums' chains; xh taken from y, which is rounded to 2^-8
    size = (1 + 2.0 ** -7) * (few.double() ** 2 / w.double()).sum(0)
    O.within(gw, fgw.double(), 2 * (LAST + 64) * O.E * size, "gw")


def test_gated_ff():
    g = torch.Generator(device=DEV).manual_seed(2)
    rows, c, f = 300000, 64, 8192
    x = torch.zeros(rows, c, dtype=BF16, device=DEV)
    x[-LAST:] = rand(g, LAST, c)
    w = rand(g, f, c) / 8, rand(g, f, c) / 8, rand(g, c, f) / 64
    y, h, kept = T.gated_ff_train(x, *w)
    gy = torch.zeros(rows, c, dtype=BF16, device=DEV)
    gy[-LAST:] = rand(g, LAST, c)
    got = [y, *T.gated_ff_backward(gy, x, *w, h, kept)]
    want = O.gated_ff(x[-LAST:], *w, "silu", gy[-LAST:])
    for n, (p, (v, bound)) in enumerate(zip(got, want)):
        if n < 2:
            assert not p[:-LAST].any()
            p = p[-LAST:]
        O.within(p, v, bound, n)


@pytest.mark.parametrize("n,c", [(8192, 64), (8, 16384)])
def test_four(n, c):
    g = torch.Generator(device=DEV).manual_seed(3)
    rows = 300000
    x = torch.zeros(rows, c, dtype=BF16, device=DEV)
    x[-LAST:] = rand(g, LAST, c)
    w = T.quantise4(rand(g, n, c) / math.sqrt(c))
    y = T.linear4(x, w)
    assert not y[:-LAST].any()
    qx, qw = O.quantise4(x[-LAST:])[2], O.unpack4(*w, c)
    want = qx @ qw.T
    O.within(y[-LAST:], want, O.U[BF16] * want.abs() + (c + 16) * O.E * (qx.abs() @ qw.abs().T) + O.TINY[BF16], "y")
    four = T.quantise4(x)
    assert not four[0][:-LAST].any() and torch.equal(T.dequantise4(four, BF16)[-LAST:].double(), qx)
