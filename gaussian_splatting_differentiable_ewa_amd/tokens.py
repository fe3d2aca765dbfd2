"""The token operators on tensors: the layers of a network that predicts
Gaussians from posed views and is trained through the rasterizer. A token stands
for one 16x16 tile of a view.

Each function checks its tensors (``ValueError``), allocates its outputs and
workspace and makes one or two calls of the C ABI on the current stream
(``_lib``); nothing is kept between calls. Token tensors are
``[batch, tokens, heads, dim]`` with any strides (views of a packed projection
need no copy); a tensor whose rows do not start on 16 bytes is copied where the
kernels need that. The functions record no graph, and refuse tensors whose
gradient would be lost that way; ``RopeAxes``, ``NormGate`` and
``BlockAttention`` are the same for ``torch.autograd``.
"""

from __future__ import annotations

from typing import Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib as L

GROUP, BLOCK = L.GS_QUERY_GROUP, L.GS_KEY_BLOCK


# The checks build their messages only when they fail, and compare device
# numbers rather than devices: small calls are bound by the host.
def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _tokens(name, t, like=None):
    if t.dim() != 4 or not t.is_cuda:
        raise ValueError(f"{name} must be [batch, tokens, heads, dim] on the GPU, got {tuple(t.shape)} on {t.device}")
    if like is not None and (t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must have the type and device of its partner")


def _vector(name, t, shape, like, dtype=torch.float32):
    if t is not None and (t.shape != shape or t.dtype is not dtype or not t.is_contiguous()
                          or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)} on {like.device}")


def _lost(form):
    """For tensors that require a gradient: refuses where one would be lost."""
    if torch.is_grad_enabled():
        raise ValueError(f"the results would carry no gradient: use {form}.apply, torch.no_grad() or detached tensors")


def _aligned(t, bytes=16):
    """t itself, or a copy, so that every row [dim] starts on that many bytes."""
    per = bytes // t.element_size()
    if t.is_contiguous() and t.data_ptr() % bytes == 0 and t.shape[3] % per == 0:
        return t
    sb, st, sh, sd = t.stride()
    b, n, h, d = t.shape
    if ((sd == 1 or d <= 1) and t.data_ptr() % bytes == 0 and (b <= 1 or sb % per == 0) and (n <= 1 or st % per == 0)
            and (h <= 1 or sh % per == 0)):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _blocks(tokens):
    return (tokens + BLOCK - 1) // BLOCK


def _groups(tokens):
    return (tokens + GROUP - 1) // GROUP


# ---- rotary positions -----------------------------------------------------------
def rope_axes(q, k, pos, freq, pairs: Sequence[int], interleaved: bool = False, inverse: bool = False):
    """Rotated q and k (k may be None). pos int32 [batch or 1, tokens, 3] (view,
    row, column), freq fp32 [dim / 2] in radians per position, pairs: the pairs
    of each axis; see gs_rope_axes."""
    _tokens("q", q)
    if q.requires_grad or k is not None and k.requires_grad:
        _lost("RopeAxes")
    b, n, hq, d = q.shape
    _need(d % 2 == 0, "dim must be even")
    if k is not None:
        _tokens("k", k, q)
        _need(k.shape[:2] == q.shape[:2] and k.shape[3] == d, "k must have q's batch, tokens and dim")
    _need(pos.dim() == 3 and pos.shape[0] in (1, b), "pos must be [batch or 1, tokens, 3]")
    _vector("pos", pos, (pos.shape[0], n, 3), q, torch.int32)
    _vector("freq", freq, (d // 2,), q)
    q = q if q.stride(3) == 1 else q.contiguous()
    q_out = torch.empty(b, n, hq, d, dtype=q.dtype, device=q.device)
    k_out = None
    if k is not None:
        k = k if k.stride(3) == 1 else k.contiguous()
        k_out = torch.empty(b, n, k.shape[2], d, dtype=q.dtype, device=q.device)
    L.gs_rope_axes(q, k, q_out, k_out, pos, freq, pairs, interleaved, inverse)
    return q_out, k_out


# ---- norms around a block -------------------------------------------------------
def _norm_args(x, f, gate, w_post, w_pre, rows_per_gate):
    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be contiguous [rows, channels] on the GPU")
    rows, c = shape = x.shape
    per = (rows or 1) if rows_per_gate is None else int(rows_per_gate)
    if per < 1:
        raise ValueError("rows_per_gate must be at least 1")
    _vector("f", f, shape, x, x.dtype)
    if gate is not None:
        _vector("gate", gate, ((rows + per - 1) // per, c), x)
    if w_post is not None:
        _vector("w_post", w_post, (c,), x)
    if w_pre is not None:
        _vector("w_pre", w_pre, (c,), x)
    if (x.requires_grad or f is not None and f.requires_grad or gate is not None and gate.requires_grad
            or w_post is not None and w_post.requires_grad or w_pre is not None and w_pre.requires_grad):
        _lost("NormGate")
    return rows, c, per


def norm_gate(x, f, gate=None, w_post=None, w_pre=None, scale: float = 1.0, eps: float = 1e-6,
              rows_per_gate: Optional[int] = None):
    """(y, h, stats): y = x + scale gate norm(f) w_post, h = norm(y) w_pre; f may
    be None (y is x then). See gs_norm_gate_fwd."""
    rows, c, per = _norm_args(x, f, gate, w_post, w_pre, rows_per_gate)
    y = x if f is None else torch.empty_like(x)
    h = torch.empty_like(x)
    stats = torch.empty(2, rows, dtype=torch.float32, device=x.device)
    L.gs_norm_gate_fwd(x, f, gate, w_post, w_pre, None if f is None else y, h, stats, per, scale, eps)
    return y, h, stats


def norm_gate_backward(gy, gh, x, f, gate, w_post, w_pre, stats, scale: float = 1.0,
                       rows_per_gate: Optional[int] = None):
    """(gx, gf, ggate, gw_post, gw_pre); None for what the forward call did not
    have. gy may be None. See gs_norm_gate_bwd."""
    rows, c, per = _norm_args(x, f, gate, w_post, w_pre, rows_per_gate)
    _vector("gy", gy, x.shape, x, x.dtype)
    _vector("gh", gh, x.shape, x, x.dtype)
    if gh.requires_grad or gy is not None and gy.requires_grad:
        _lost("NormGate")
    _vector("stats", stats, (2, rows), x)
    gx = torch.empty_like(x)
    gf = None if f is None else torch.empty_like(x)
    ggate = None if gate is None or f is None else torch.empty_like(gate)
    gw_post = None if w_post is None or f is None else torch.empty_like(w_post)
    gw_pre = None if w_pre is None else torch.empty_like(w_pre)
    ws = torch.empty(L.norm_gate_bwd_workspace_bytes(rows, c, per), dtype=torch.uint8, device=x.device)
    L.gs_norm_gate_bwd(gy, gh, x, f, gate, w_post, w_pre, stats, gx, gf, ggate, gw_post, gw_pre, per, ws, scale)
    return gx, gf, ggate, gw_post, gw_pre


# ---- choice of key blocks -------------------------------------------------------
def _length(kv_len, q):
    _vector("kv_len", kv_len, (q.shape[0],), q, torch.int32)


def _summary(name, s, shape, like):
    sum8, scale = s
    if (sum8.shape != shape or sum8.dtype is not torch.int8 or scale.shape != shape[:3] or scale.dtype is not torch.float32
            or sum8.get_device() != like.get_device() or scale.get_device() != like.get_device()
            or (sum8.stride(3) != 1 and shape[3] > 1)):
        raise ValueError(f"{name} must be int8 {shape} (its last dimension contiguous) and float32 {shape[:3]} on "
                         f"{like.device}")


def block_summary(k, kv_len=None, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, block0: int = 0,
                  blocks: Optional[int] = None):
    """(sum8, scale) of the keys' blocks of 64, or of `blocks` of them (the rest)
    from block0 on written into `out` (a growing cache renews its last blocks).
    The means are in steps of 2^-8: for keys of order one. See gs_block_summary."""
    _tokens("k", k)
    _length(kv_len, k)
    b, n, h, d = k.shape
    if out is None:
        _need(block0 == 0 and blocks is None, "block0 and blocks need out")
        out = (torch.empty(b, h, _blocks(n), d, dtype=torch.int8, device=k.device),
               torch.empty(b, h, _blocks(n), dtype=torch.float32, device=k.device))
    _summary("out", out, (b, h, _blocks(n), d), k)
    L.gs_block_summary(_aligned(k), out[0], out[1], kv_len, block0, blocks)
    return out


def select_blocks(q, summary, tokens_k: int, top: int, kv_len=None, causal: bool = False):
    """int32 [batch, heads, ceil(tokens / 128), top]: the key blocks of every group
    of 128 queries, ascending, -1 after the last. See gs_block_select."""
    _tokens("q", q)
    _length(kv_len, q)
    b, n, h, d = q.shape
    sum8, scale = summary
    _need(sum8.dim() == 4, "summary must be block_summary's")
    hk = sum8.shape[1]
    _need(hk > 0 and h % hk == 0, "q's heads must be a multiple of the summary's")
    _summary("summary", summary, (b, hk, _blocks(tokens_k), d), q)
    lists = torch.empty(b, h, _groups(n), top, dtype=torch.int32, device=q.device)
    L.gs_block_select(_aligned(q), _aligned(sum8, 8), scale, tokens_k, hk, lists, kv_len, causal)
    return lists


# ---- attention over the chosen blocks -------------------------------------------
def _attn_args(q, k, v, lists, kv_len):
    _tokens("q", q)
    _tokens("k", k, q)
    _tokens("v", v, q)
    b, n, h, d = q.shape
    kb, _, hk, kd = k.shape
    if kb != b or kd != d or v.shape != k.shape:
        raise ValueError("k and v must have q's batch and dim")
    if hk == 0 or h % hk != 0:
        raise ValueError("q's heads must be a multiple of k's")
    if lists.dim() != 4:
        raise ValueError("lists must be [batch, heads, groups, top]")
    _vector("lists", lists, (b, h, _groups(n), lists.shape[3]), q, torch.int32)
    _length(kv_len, q)
    if q.requires_grad or k.requires_grad or v.requires_grad:
        _lost("BlockAttention")


def block_attention(q, k, v, lists, sm_scale: Optional[float] = None, kv_len=None, causal: bool = False):
    """(out, lse): attention of each query over its group's listed key blocks;
    fp16 or bf16, dim 64 or 128. causal: the last query is the last key (of
    kv_len); sequences padded on the right for training take no kv_len. See
    gs_block_attn_fwd."""
    _attn_args(q, k, v, lists, kv_len)
    b, n, h, d = q.shape
    out = torch.empty(b, n, h, d, dtype=q.dtype, device=q.device)
    lse = torch.empty(b, h, n, dtype=torch.float32, device=q.device)
    need = L.block_attn_fwd_workspace_bytes(b, n, h, d, lists.shape[3])
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    L.gs_block_attn_fwd(_aligned(q), _aligned(k), _aligned(v), lists, out, lse, ws, kv_len, causal, sm_scale)
    return out, lse


def block_attention_backward(gout, q, k, v, out, lse, lists, sm_scale: Optional[float] = None, kv_len=None,
                             causal: bool = False):
    """(gq, gk, gv) of block_attention; in fp16 the scores' gradients have to fit
    the type. See gs_block_attn_bwd."""
    _attn_args(q, k, v, lists, kv_len)
    _tokens("gout", gout, q)
    _tokens("out", out, q)
    if gout.requires_grad or out.requires_grad:
        _lost("BlockAttention")
    _need(gout.shape == q.shape and out.shape == q.shape, "gout and out must have q's shape")
    b, n, h, d = q.shape
    _vector("lse", lse, (b, h, n), q)
    m, hk = k.shape[1:3]
    gq = torch.empty(b, n, h, d, dtype=q.dtype, device=q.device)
    gk = torch.empty(b, m, hk, d, dtype=q.dtype, device=q.device)
    gv = torch.empty(b, m, hk, d, dtype=q.dtype, device=q.device)
    need = L.block_attn_bwd_workspace_bytes(b, n, m, h, hk, d)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    L.gs_block_attn_bwd(_aligned(gout), _aligned(q), _aligned(k), _aligned(v), _aligned(out), lse, lists, gq, gk, gv, ws,
                        kv_len, causal, sm_scale)
    return gq, gk, gv


# ---- for torch.autograd ---------------------------------------------------------
# Differentiable once: the backward kernels record no graph, so a gradient of
# their gradients (create_graph=True) raises instead of lacking their part.
class RopeAxes(torch.autograd.Function):
    """apply(q, k, pos, freq, pairs, interleaved=False) -> q', k' (gradients of q
    and k only)."""

    @staticmethod
    def forward(ctx, q, k, pos, freq, pairs, interleaved=False):
        ctx.save_for_backward(pos, freq)
        ctx.how = (pairs, interleaved)
        return rope_axes(q, k, pos, freq, pairs, interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, gq, gk):
        pos, freq = ctx.saved_tensors
        gq, gk = rope_axes(gq, gk, pos, freq, ctx.how[0], ctx.how[1], inverse=True)
        return gq, gk, None, None, None, None


class NormGate(torch.autograd.Function):
    """apply(x, f, gate, w_post, w_pre, scale=1, eps=1e-6, rows_per_gate=None) ->
    y, h. Without f, y is x and only the norm is differentiated through h."""

    @staticmethod
    def forward(ctx, x, f, gate, w_post, w_pre, scale=1.0, eps=1e-6, rows_per_gate=None):
        y, h, stats = norm_gate(x, f, gate, w_post, w_pre, scale, eps, rows_per_gate)
        ctx.save_for_backward(x, f, gate, w_post, w_pre, stats)
        ctx.how = (scale, rows_per_gate)
        return (x.view_as(x) if f is None else y), h

    @staticmethod
    @once_differentiable
    def backward(ctx, gy, gh):
        gy = None if gy is None else gy.contiguous()
        grads = norm_gate_backward(gy, gh.contiguous(), *ctx.saved_tensors, scale=ctx.how[0], rows_per_gate=ctx.how[1])
        return (*grads, None, None, None)


class BlockAttention(torch.autograd.Function):
    """apply(q, k, v, lists, sm_scale=None, kv_len=None, causal=False) -> out."""

    @staticmethod
    def forward(ctx, q, k, v, lists, sm_scale=None, kv_len=None, causal=False):
        out, lse = block_attention(q, k, v, lists, sm_scale, kv_len, causal)
        ctx.save_for_backward(q, k, v, out, lse, lists, kv_len)
        ctx.how = (sm_scale, causal)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, gout):
        q, k, v, out, lse, lists, kv_len = ctx.saved_tensors
        grads = block_attention_backward(gout, q, k, v, out, lse, lists, ctx.how[0], kv_len, ctx.how[1])
        return (*grads, None, None, None, None)
