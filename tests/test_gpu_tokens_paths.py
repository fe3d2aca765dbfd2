"""The token operators past the sizes at which their kernels go over to another
form or refill what they hold: against the same 64-bit definitions."""

import pytest
import torch

import test_gpu_tokens as base
import token_oracle as O
from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("b,lq,lk,hq,hk,d,top,cut", [
    (1, 300, 19200, 100, 4, 128, 20, None),           # 300 lists of 300 blocks: one wave a list, several scores a lane
    (2, 300, 19200, 50, 5, 64, 30, (19200, 17001)),
    (1, 300, 19200, 100, 4, 40, 7, None),             # no 64 dimensions at a time
    (1, 300, 44800, 100, 4, 64, 33, None),            # 300 lists of 700 blocks: four waves a list
    (1, 300, 44800, 100, 2, 256, 33, (44700,)),
    (1, 2, 192000, 3, 1, 64, 50, None),               # sixteen waves, three rounds of them
    (1, 130, 4160, 1, 1, 64, 50, None),
])
def test_select_by_every_number_of_waves(causal, b, lq, lk, hq, hk, d, top, cut):
    g = base.gen(lk + d)
    q, k = base.rand(g, b, lq, hq, d, dtype=BF16), base.rand(g, b, lk, hk, d, dtype=BF16)
    length = None if cut is None else torch.tensor(cut, dtype=torch.int32, device="cuda")
    eight, scale = T.block_summary(k, length)
    got = T.select_blocks(q, (eight, scale), lk, top, length, causal)
    assert torch.equal(got.cpu(), O.select(q, (eight.long(), scale.double()), lk, top, length, causal))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lq,lk,hq,d,top", [
    (4300, 1000, 2, 64, 6),     # over 32 groups: a second word of each block's bits
    (4300, 4300, 2, 128, 6),
    (4300, 700, 34, 64, 3),     # 68 words a block: the walk refills
])
def test_backward_over_many_groups(causal, lq, lk, hq, d, top):
    g = base.gen(lq + lk)
    q, gout = (base.rand(g, 1, lq, hq, d, dtype=BF16) for _ in range(2))
    k, v = (base.rand(g, 1, lk, 1, d, dtype=BF16) for _ in range(2))
    lists = base.random_lists(g, 1, hq, (lq + 127) // 128, (lk + 63) // 64, top)
    base.check_attention(q, k, v, lists, gout, None, causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("hq,d", [(2, 64), (100, 64), (50, 128)])
def test_lists_of_more_than_64_blocks(causal, hq, d):
    g = base.gen(hq)
    q, gout = (base.rand(g, 1, 200, hq, d, dtype=F16) for _ in range(2))
    k, v = (base.rand(g, 1, 8320, 2, d, dtype=F16) for _ in range(2))
    lists = base.random_lists(g, 1, hq, 2, 130, 100)
    base.check_attention(q, k, v, lists, gout, None, causal)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,c,per", [(9000, 72, 100), (9000, 256, 7), (8300, 250, 65), (5000, 1027, 600), (4200, 2048, 4)])
def test_norms_of_many_rows_and_gates(dtype, rows, c, per):
    """More than one row a run, gates that change inside one, more than 64 gates."""
    base.test_norm_gate(dtype, rows, c, per, "fgw")
    base.test_norm_gate_backward(dtype, rows, c, per, "fgw", True)


def test_backward_with_large_scores_and_values():
    """Scores of several hundred, and values near the type's largest with
    output gradients that keep gout . v inside it."""
    for dtype, big in ((F16, 3e4), (BF16, 1e30)):
        g = base.gen(6)
        q, k, v, gout = (base.rand(g, 1, 140, 2, 64, dtype=dtype) for _ in range(4))
        lists = base.random_lists(g, 1, 2, 2, 3, 3)
        base.check_attention(30 * q, 3 * k, v, lists, gout, None, True, scale=0.5)
        wide = (v.float() * (big / v.abs().max().float())).to(dtype)
        base.check_attention(q, k, wide, lists, (gout.float() * (1000 / big)).to(dtype), None, False)
