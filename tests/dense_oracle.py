"""Layer norm, the gated feed-forward block and 4-bit linear layers from their
definitions in 64 bits, for the GPU tests, with what their error bounds are made
of: the sums of magnitudes that roundings are relative to."""

import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half an ulp, relative
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the least subnormal
E = 2.0 ** -24


def within(got, want, bound, what):
    """Every element within its bound; what is not finite, the same."""
    got, fine = got.double(), torch.isfinite(want)
    assert got.shape == want.shape, what
    assert torch.equal(torch.isfinite(got), fine), f"{what}: other elements are finite"
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: other elements are NaN"
    over = ((got - want).abs() - bound)[fine]
    assert over.numel() == 0 or over.max() <= 0, f"{what}: {over.max().item():.3e} over the bound"


def layer_norm(x, w, b, eps):
    x = x.double()
    x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())


def layer_norm_gradients(gy, x, w, eps):
    """gx, gw, gb and the magnitudes that their roundings are relative to."""
    x, gy = x.double(), gy.double()
    w = torch.ones(x.shape[1], dtype=torch.double, device=x.device) if w is None else w.double()
    x0 = x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((x0 * x0).mean(-1, keepdim=True) + eps)
    xh, d = x0 * r, gy * w
    gx = r * (d - d.mean(-1, keepdim=True) - xh * (d * xh).mean(-1, keepdim=True))
    # xh is off by roundings of the mean of x too
    mag = xh.abs() + r * x.abs().mean(-1, keepdim=True)
    d = d.abs()
    return ((gx, r * (d + d.mean(-1, keepdim=True) + mag * (d * mag).mean(-1, keepdim=True))),
            ((gy * xh).sum(0), (gy.abs() * mag).sum(0)), (gy.sum(0), gy.abs().sum(0)))
