"""Training on sequences of several lengths, padded on the right: causal
attention without a key length, as gs.h says, is each sequence's own."""

import pytest
import torch

import token_oracle as O
from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("heads", [4, 72])
def test_right_padded_sequences(dtype, d, heads):
    g = torch.Generator(device="cuda").manual_seed(d)
    n, lengths = 384, (384, 250, 1)
    q, gout = (torch.randn(3, n, heads, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    k, v = (torch.randn(3, n, 2, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    for i, m in enumerate(lengths):
        gout[i, m:] = 0  # the loss does not look at the padding
    sums = T.block_summary(k, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    lists = T.select_blocks(q, sums, n, 3, None, True)
    q, k, v = (t.requires_grad_() for t in (q, k, v))
    out = T.BlockAttention.apply(q, k, v, lists, None, None, True)
    out.backward(gout)
    for i, m in enumerate(lengths):
        one = slice(i, i + 1)
        groups = (m + 127) // 128
        want, bound = O.attention(*(t.detach()[one, :m] for t in (q, k, v)), lists[one, :, :groups], d ** -0.5, None, True,
                                  gout[one, :m])
        for name, x in (("out", out.detach()), ("gq", q.grad), ("gk", k.grad), ("gv", v.grad)):
            assert ((x[one, :m].double() - want[name]).abs() <= bound[name]).all(), (i, name)
            if name != "out":
                assert not x[one, m:].any(), (i, name)
