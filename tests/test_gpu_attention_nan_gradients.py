"""A NaN in a query reaches its own row of gq, not its neighbours'."""

import pytest
import torch

import token_oracle as O
from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", ["q", "gout"])
def test_nan_query_gradient(dtype, d, bad):
    g = torch.Generator(device="cuda").manual_seed(d)
    q, gout = (torch.randn(1, 150, 2, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    k, v = (torch.randn(1, 700, 1, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    lists = T.select_blocks(q, T.block_summary(k), 700, 4)
    want, bound = O.attention(q, k, v, lists, d ** -0.5, gout=gout)
    (q if bad == "q" else gout)[0, 37, 1, 5] = float("nan")
    out, lse = T.block_attention(q, k, v, lists)
    gq, gk, gv = T.block_attention_backward(gout, q, k, v, out, lse, lists)
    here = torch.ones(150, 2, dtype=torch.bool, device="cuda")
    here[37, 1] = False
    assert torch.isnan(gq[0, 37, 1]).all()
    assert ((gq.double() - want["gq"]).abs() <= bound["gq"])[0][here].all()
    # keys that the row's group does not list have no part in it
    listed = torch.zeros(11, dtype=torch.bool, device="cuda")
    listed[lists[0, 1, 0].long()] = True
    away = ~listed.repeat_interleave(64)[:700]
    for x, name in ((gk, "gk"), (gv, "gv")):
        assert ((x.double() - want[name]).abs() <= bound[name])[0, away].all()
        assert torch.isnan(x[0, ~away]).any()
