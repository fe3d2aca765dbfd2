"""The gated feed-forward block in the tiles and splits that other tests' sizes
do not take, against its definition in 64 bits."""

import pytest
import torch

import dense_oracle as O
from gaussian_splatting_differentiable_ewa_amd import tokens as T
from test_gpu_gated_ff import BF16, F16, NAMES, case, gen

pytestmark = pytest.mark.gpu

# what each is for, by product (h, y, gg and gu), tile and whether the sum is split; on and off the tiles
SIZES = [(2048, 512, 1024, 512), (1500, 512, 1024, 512), (132, 8, 5704, 8),  # h, 128
         (3600, 256, 1024, 256), (10893, 16, 136, 8),  # gg and gu, 128
         (72, 6056, 2104, 120), (648, 6856, 1504, 40),  # h, 128 and 256, split
         (70, 48, 5976, 4184), (736, 16, 7904, 2712),  # y, 128 and 256, split
         (4236, 24, 72, 6536), (1759, 32, 1160, 6208)]  # gg and gu, 128 and 256, split


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,c,f,co", SIZES)
def test_both_ways(dtype, act, rows, c, f, co):
    x, wg, wu, wd, gy = case(gen(rows + c), rows, c, f, co, dtype)
    want = O.gated_ff(x, wg, wu, wd, act, gy)
    y, h, kept = T.gated_ff_train(x, wg, wu, wd, act)
    got = [y, *T.gated_ff_backward(gy, x, wg, wu, wd, h, kept, act)]
    for name, p, (w, bound) in zip(NAMES, got, want):
        O.within(p, w, bound, name)
    # h alone, where no kept bits go out, is formed by the same tiles
    assert torch.equal(T.gated_ff(x, wg, wu, wd, act), y)
