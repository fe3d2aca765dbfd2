"""A NaN in a query reaches its own row of the outputs, and only that: such a row
must not look like one that sees no key (zeros and -infinity)."""

import math

import pytest
import torch

import token_oracle as O
from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,heads,top", [(1, 2, 24), (5, 1, 2), (130, 100, 3)], ids=["split", "few", "full groups"])
def test_nan_query(dtype, d, n, heads, top):
    g = torch.Generator(device="cuda").manual_seed(n)
    q = torch.randn(1, n, heads, d, generator=g, device="cuda").to(dtype)
    k, v = (torch.randn(1, 2000, 1, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    lists = T.select_blocks(q, T.block_summary(k), 2000, top)
    lists[0, heads - 1] = lists[0, 0]
    want, bound = O.attention(q, k, v, lists, d ** -0.5)
    q[0, n - 1, heads - 1] = float("nan")
    out, lse = T.block_attention(q, k, v, lists)
    assert torch.isnan(out[0, n - 1, heads - 1]).all() and torch.isnan(lse[0, heads - 1, n - 1])
    here = torch.ones(n, heads, dtype=torch.bool, device="cuda")
    here[n - 1, heads - 1] = False
    assert ((out.double() - want["out"]).abs() <= bound["out"])[0][here].all()
    assert ((lse.double() - want["lse"]).abs() <= bound["lse"])[0].T[here].all()
    # one that sees no key stays zeros and -infinity, whatever its query holds
    lists[0, heads - 1, -1] = -1
    out, lse = T.block_attention(q, k, v, lists)
    assert not out[0, n - 1, heads - 1].any() and lse[0, heads - 1, n - 1] == -math.inf
