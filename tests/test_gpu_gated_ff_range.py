"""The range of the gated feed-forward block's hidden layer: fp16 holds |h| up to
65504, and a row with more than that is not finite; bf16 holds it."""

import math

import pytest
import torch

import dense_oracle as O
from gaussian_splatting_differentiable_ewa_amd import tokens as T
from test_gpu_gated_ff import BF16, DEV, F16, NAMES, case, gen

pytestmark = pytest.mark.gpu


def hidden(act, x, wg, wu):
    return O.activation(act, x.double() @ wg.double().T)[0] * (x.double() @ wu.double().T)


# few rows; tiles; the sum of h in splits
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,c,f,co", [(16, 64, 64, 64), (300, 64, 64, 64), (66, 2048, 256, 64)])
def test_rows_around_the_largest_of_fp16(act, rows, c, f, co):
    x, wg, wu, wd, gy = case(gen(rows), rows, c, f, co, F16)
    wd = wd / 64  # y stays in the type where h does not
    # every other row's largest |h| to just below 65504, the others' from there up to 64 times as much: h grows with
    # the square of x where the gate is open, which it is for the largest from the first step on
    at = torch.arange(rows, device=DEV)
    target = torch.where(at % 2 == 0, 0.99, 1.01 * 64.0 ** (at / rows)) * 65504
    x = x.double() * 64
    for _ in range(4):
        x = x * (target / hidden(act, x, wg, wu).abs().amax(1)).sqrt()[:, None]
    x = x.to(F16)
    h = hidden(act, x, wg, wu)
    most = h.abs().amax(1)
    fits, over = most < 65504, most > 65520 * (1 + 2.0 ** -10)
    assert fits.sum() > rows // 4 and over.sum() > rows // 4 and (fits & (most > 32000)).any()
    want = O.gated_ff(x, wg, wu, wd, act, gy)
    assert torch.isfinite(want[0][0].half()).all()
    y, hid, kept = T.gated_ff_train(x, wg, wu, wd, act)
    O.within(y[fits], want[0][0][fits], want[0][1][fits], "y")
    assert not torch.isfinite(y[over]).all(1).any()
    assert torch.equal(T.gated_ff(x, wg, wu, wd, act).view(torch.int16), y.view(torch.int16))
    # rows that fit, by themselves, both ways
    x, gy = x[fits].contiguous(), (gy[fits] / 4096).contiguous()
    want = O.gated_ff(x, wg, wu, wd, act, gy)
    y, hid, kept = T.gated_ff_train(x, wg, wu, wd, act)
    for name, p, (w, bound) in zip(NAMES, [y, *T.gated_ff_backward(gy, x, wg, wu, wd, hid, kept, act)], want):
        O.within(p, w, bound, name)
    assert math.isfinite(float(hid.float().abs().max())) and float(hid.float().abs().max()) > 32000


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_bf16_holds_them(act):
    x, wg, wu, wd, gy = case(gen(1), 70, 64, 64, 64, BF16)
    x = x * 256
    want = O.gated_ff(x, wg, wu, wd, act, gy)
    y, hid, kept = T.gated_ff_train(x, wg, wu, wd, act)
    assert float(hid.float().abs().max()) > 65536
    for name, p, (w, bound) in zip(NAMES, [y, *T.gated_ff_backward(gy, x, wg, wu, wd, hid, kept, act)], want):
        O.within(p, w, bound, name)
