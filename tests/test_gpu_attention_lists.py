"""Lists that come back to a block: an entry counts only if it exceeds every
entry before it, in both directions and in both forward kernels."""

import pytest
import torch

from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = pytest.mark.gpu


def strict(rows):
    """The same lists with the entries that do not count replaced by -1."""
    out = []
    for row in rows:
        most, kept = -1, []
        for m in row:
            kept.append(m if m > most else -1)
            most = max(most, m)
        out.append(kept)
    return out


SHORT = [[5, 3, 5, -1, 6, 6], [1, 0, 1, 2, 1, 4], [2, -1, 2, -7, 3, 0], [4, 4, 3, 4, 5, 2]]


def long_list():
    """Over 64 entries, with a repeat of an entry far before it on either side of the 64th."""
    row = list(range(0, 140, 2))
    row[10], row[63], row[64], row[66] = 4, 30, 126, 8
    return [row, row[::-1], [-1] * 63 + [9, 3, 9, 11, 9, 11, 12], [6] + [-1] * 64 + [6, 2, 7, 6, 7]]


@pytest.mark.parametrize("rows,blocks", [(SHORT, 7), (long_list(), 140)], ids=["short", "past 64 entries"])
@pytest.mark.parametrize("heads", [2, 100], ids=["split lists", "full groups"])
@pytest.mark.parametrize("causal", [False, True])
def test_entries_that_do_not_ascend_are_skipped(rows, blocks, heads, causal):
    g = torch.Generator(device="cuda").manual_seed(blocks)
    n, d, lk = 250, 64, blocks * 64 - 5
    q, gout = (torch.randn(1, n, heads, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn(1, lk, 2, d, generator=g, device="cuda").bfloat16() for _ in range(2))

    def lists(r):
        t = torch.tensor(r, dtype=torch.int32, device="cuda").view(1, 2, 2, -1)
        return t.repeat_interleave(heads // 2, 1).contiguous()

    got, clean = lists(rows), lists(strict(rows))
    assert not torch.equal(got, clean)
    out, lse = T.block_attention(q, k, v, got, causal=causal)
    want = T.block_attention(q, k, v, clean, causal=causal)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    grads = T.block_attention_backward(gout, q, k, v, out, lse, got, causal=causal)
    for x, y in zip(grads, T.block_attention_backward(gout, q, k, v, *want, clean, causal=causal)):
        assert torch.equal(x, y)
