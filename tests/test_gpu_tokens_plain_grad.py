"""The plain functions record no gradient: where one would be lost they refuse."""

import pytest
import torch

from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def rand(*shape, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(len(shape)), device="cuda").to(dtype)


def calls():
    """Name, call, tensors whose gradient it would lose."""
    q, k, v = (rand(1, 70, 2, 64) for _ in range(3))
    pos, freq = torch.ones(1, 70, 3, dtype=torch.int32, device="cuda"), rand(32, dtype=torch.float32).abs()
    lists = torch.tensor([0, 1], dtype=torch.int32, device="cuda").expand(1, 2, 1, 2).contiguous()
    out, lse = T.block_attention(q, k, v, lists)
    x, f = rand(6, 64), rand(6, 64)
    gate, w2, w1 = (rand(*s, dtype=torch.float32) for s in ((1, 64), (64,), (64,)))
    stats = T.norm_gate(x, f, gate, w2, w1)[2]
    return [("rope_axes", lambda: T.rope_axes(q, k, pos, freq, (8, 12, 12)), (q, k)),
            ("norm_gate", lambda: T.norm_gate(x, f, gate, w2, w1), (x, f, gate, w2, w1)),
            ("norm_gate_backward", lambda: T.norm_gate_backward(x, f, x, f, gate, w2, w1, stats), (x, f, gate, w2, w1)),
            ("block_attention", lambda: T.block_attention(q, k, v, lists), (q, k, v)),
            ("block_attention_backward", lambda: T.block_attention_backward(out, q, k, v, out, lse, lists), (out, q, k, v))]


def test_plain_functions_refuse_to_lose_a_gradient():
    for name, call, tensors in calls():
        call()
        for t in tensors:
            t.requires_grad_()
            with pytest.raises(ValueError, match="gradient"):
                call()
            with torch.no_grad():
                call()
            t.requires_grad_(False)


def test_a_layer_keeps_the_gradients_of_its_projections():
    """A layer in training: every weight before the attention learns."""
    h = rand(1, 200, 64)
    # scores of order one: a saturated softmax has no gradient to lose
    weights = list((rand(3, 64, 128) / 16).unbind(0))
    for w in weights:
        w.requires_grad_()
    q, k, v = ((h @ w).view(1, 200, 2, 64) for w in weights)
    pos = torch.arange(200, device="cuda").int()[None, :, None].expand(1, 200, 3).contiguous()
    freq = 100.0 ** -(torch.arange(32, device="cuda") / 32)
    q, k = T.RopeAxes.apply(q, k, pos, freq, (8, 12, 12))
    lists = T.select_blocks(q, T.block_summary(k), k.shape[1], top=2)  # whole numbers: no gradient to lose
    T.BlockAttention.apply(q, k, v, lists).float().pow(2).sum().backward()
    assert all(w.grad is not None and w.grad.any() for w in weights)
