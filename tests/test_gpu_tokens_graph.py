"""The token operators captured in a graph: every replay gives the eager bits,
with new inputs in the captured buffers and eager work between the replays."""

import pytest
import torch

from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,lk,heads,d", [(1, 3000, 4, 128), (300, 700, 4, 64), (1500, 1500, 12, 128)],
                         ids=["split lists", "few", "full groups"])
def test_replays_equal_eager_calls(n, lk, heads, d):
    def inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        pos = torch.randint(0, 99, (1, lk, 3), generator=g, device="cuda").int()
        return [r(1, lk, heads, d).bfloat16(), r(1, lk, 2, d).bfloat16(), r(1, lk, 2, d).bfloat16(), r(n, 256).bfloat16(),
                r(n, 256).bfloat16(), r((n + 99) // 100, 256), r(256), pos, r(d // 2).abs(),
                torch.randint(lk // 2, lk + 1, (1,), generator=g, device="cuda").int(), r(1, lk, heads, d).bfloat16()]

    def run(t):
        """One layer's operators, forward and backward; the queries are the last n tokens."""
        q, _ = T.rope_axes(t[0][:, lk - n:], None, t[7][:, lk - n:].contiguous(), t[8], (d // 8, 0, d // 8))
        k, _ = T.rope_axes(t[1], None, t[7], t[8], (d // 8, 0, d // 8), True)
        sums = T.block_summary(k, t[9])
        lists = T.select_blocks(q, sums, lk, 5, t[9], True)
        out, lse = T.block_attention(q, k, t[2], lists, None, t[9], True)
        grads = T.block_attention_backward(t[10][:, lk - n:], q, k, t[2], out, lse, lists, None, t[9], True)
        x, f, gate, w = t[3:7]
        y, h, stats = T.norm_gate(x, f, gate, w, w, 0.5, 1e-6, 100)
        return [q, k, *sums, lists, out, lse, *grads, y, h,
                *T.norm_gate_backward(y, h, x, f, gate, w, w, stats, 0.5, 100)]

    held = inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = run(held)
    for seed in (0, 1, 2, 3):
        fresh = inputs(seed)
        for t, u in zip(held, fresh):
            t.copy_(u)
        graph.replay()
        got = [t.clone() for t in results]
        torch.cuda.synchronize()
        for x, y in zip(got, run(fresh)):
            assert torch.equal(x.flatten().view(torch.uint8), y.flatten().view(torch.uint8)), seed
