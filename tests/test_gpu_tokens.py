"""The token operators on the GPU against their definitions in 64 bits."""

import math

import pytest
import torch

import token_oracle as O
from gaussian_splatting_differentiable_ewa_amd import _lib as L
from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
DEV = "cuda"


def gen(seed=0):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def within(got, want, bound, what):
    """Every element within its bound; infinities and zeros of empty rows exactly."""
    got, fine = got.double(), torch.isfinite(want)
    assert got.shape == want.shape, what
    assert torch.equal(torch.isfinite(got), fine), f"{what}: other elements are finite"
    assert torch.equal(got[~fine], want[~fine]), f"{what}: infinities differ"
    over = ((got - want).abs() - bound)[fine]
    assert over.numel() == 0 or over.max() <= 0, f"{what}: {over.max().item():.3e} over the bound"


# ---- rotary positions -----------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("b,n,hq,hk,d,pairs,interleaved", [
    (1, 1, 1, 0, 2, (1, 0, 0), False),
    (2, 7, 3, 1, 64, (8, 12, 12), False),
    (1, 129, 5, 5, 128, (16, 20, 20), True),   # some pairs unrotated
    (2, 33, 2, 1, 30, (5, 5, 5), False),        # no 16-byte accesses
    (1, 40, 9, 2, 96, (0, 48, 0), True),
    (1, 5, 2, 2, 64, (0, 0, 0), False),         # a copy
])
def test_rope(dtype, inverse, b, n, hq, hk, d, pairs, interleaved):
    g = gen(n)
    q, k = rand(g, b, n, hq, d, dtype=dtype), (rand(g, b, n, hk, d, dtype=dtype) if hk else None)
    pos = torch.randint(0, 5000, (b, n, 3), generator=g, device=DEV, dtype=torch.int32)
    freq = 10000.0 ** -torch.rand(d // 2, generator=g, device=DEV)
    got = T.rope_axes(q, k, pos, freq, pairs, interleaved, inverse)
    for x, y in zip((q, k), got):
        if x is None:
            assert y is None
            continue
        want, mag = O.rope(x, pos, freq, pairs, interleaved, inverse)
        # sine and cosine 2 ulp, the carried product's second order, two products and a sum
        within(y, want, O.U[dtype] * want.abs() + 8 * O.E * mag + O.TINY[dtype], "rope")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rope_strides_in_place_and_back(dtype):
    """A packed projection, a transposed layout, a misaligned slice and in-place
    calls; the inverse undoes the rotation."""
    g = gen(3)
    packed = rand(g, 2, 19, (4 + 2 + 2) * 64 + 1, dtype=dtype)
    for first in (0, 1):  # 1: rows off 16 bytes
        q = packed[..., first: first + 256].unflatten(-1, (4, 64))
        k = packed[..., first + 256: first + 384].unflatten(-1, (2, 64))
        pos = torch.randint(-9, 99, (1, 19, 3), generator=g, device=DEV, dtype=torch.int32)
        freq = torch.rand(32, generator=g, device=DEV)
        got = T.rope_axes(q, k, pos, freq, (10, 11, 11))
        for x, y in zip((q, k), got):
            want, mag = O.rope(x, pos.expand(2, -1, -1), freq, (10, 11, 11), False, False)
            within(y, want, O.U[dtype] * want.abs() + 8 * O.E * mag, "rope strided")
        turned = packed.clone()
        qt, kt = turned[..., first: first + 256].unflatten(-1, (4, 64)), turned[..., first + 256: first + 384].unflatten(-1, (2, 64))
        L.gs_rope_axes(qt, kt, qt, kt, pos, freq, (10, 11, 11))
        assert torch.equal(qt, got[0]) and torch.equal(kt, got[1])
        assert torch.equal(turned[..., first + 384:], packed[..., first + 384:])
        heads_first = q.transpose(1, 2).contiguous().transpose(1, 2)
        assert torch.equal(T.rope_axes(heads_first, None, pos, freq, (10, 11, 11))[0], got[0])
        back = T.rope_axes(*got, pos, freq, (10, 11, 11), inverse=True)[0]
        mag = O.rope(q, pos.expand(2, -1, -1), freq, (10, 11, 11), False, False)[1]
        within(back, q.double(), (3 * O.U[dtype] + 16 * O.E) * mag, "rope back")


def test_rope_gradient():
    """<rope(x), y> differentiated by x, against the formula and against
    differences of the 64-bit form."""
    g = gen(5)
    q, k = rand(g, 1, 9, 2, 32).requires_grad_(), rand(g, 1, 9, 2, 32).requires_grad_()
    pos = torch.randint(0, 50, (1, 9, 3), generator=g, device=DEV, dtype=torch.int32)
    freq = torch.rand(16, generator=g, device=DEV)
    yq, yk = rand(g, 1, 9, 2, 32), rand(g, 1, 9, 2, 32)
    qo, ko = T.RopeAxes.apply(q, k, pos, freq, (4, 6, 6), True)
    ((qo * yq).sum() + (ko * yk).sum()).backward()
    for x, y in ((q, yq), (k, yk)):
        want, mag = O.rope(y, pos, freq, (4, 6, 6), True, True)
        within(x.grad, want, 16 * O.E * mag, "rope gradient")
        dx, step = rand(g, 1, 9, 2, 32).double(), 1e-3
        f = lambda s: (O.rope(x.detach().double() + s * dx, pos, freq, (4, 6, 6), True, False)[0] * y).sum()  # noqa: E731,B023
        slope = ((f(step) - f(-step)) / (2 * step)).item()
        assert abs((x.grad.double() * dx).sum().item() - slope) <= 16 * O.E * (mag * dx.abs()).sum().item() + 1e-9


# ---- norms around a block -------------------------------------------------------
def _norm_case(g, rows, c, per, dtype, parts):
    x, f = rand(g, rows, c, dtype=dtype), rand(g, rows, c, dtype=dtype)
    gate = rand(g, (rows + per - 1) // per, c) if "g" in parts else None
    w2 = 1 + 0.3 * rand(g, c) if "w" in parts else None
    w1 = 1 + 0.3 * rand(g, c) if "w" in parts else None
    return x, (f if "f" in parts else None), gate, w2, w1


NORM_SIZES = [(1, 1, 1), (1, 64, 1), (7, 96, 3), (130, 250, 50), (65, 512, 65), (33, 1000, 8), (40, 1027, 9), (9, 2048, 4),
              (5, 4096, 2), (6, 3000, 6), (3, 5001, 1), (3, 8192, 3), (2, 16384, 1), (2, 16383, 2), (3000, 72, 700)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,c,per", NORM_SIZES)
@pytest.mark.parametrize("parts", ["fgw", "fw", "f", "w", ""])
def test_norm_gate(dtype, rows, c, per, parts):
    if "f" not in parts and "g" in parts:
        pytest.skip("a gate needs f")
    g = gen(c)
    x, f, gate, w2, w1 = _norm_case(g, rows, c, per, dtype, parts)
    eps, a = 1e-5, 0.6
    y, h, stats = T.norm_gate(x, f, gate, w2, w1, a, eps, per)
    wy, wh = O.norm_gate(x, f, gate, w2, w1, a, eps, per)
    # a sum of c squares in fp32 is off by at most (c / 64 + 12) roundings along its longest chain, 1 / sqrt halves that
    rel = (c / 64 + 24) * O.E
    mag = x.double().abs() + (wy - x.double()).abs()
    within(y, wy, O.U[dtype] * wy.abs() * (f is not None) + rel * mag + O.TINY[dtype], "y")
    r1 = 1 / torch.sqrt((wy * wy).mean(-1, keepdim=True) + eps)
    wmag = mag * r1 * (1 if w1 is None else w1.double().abs())
    within(h, wh, O.U[dtype] * wh.abs() + 3 * rel * wmag + rel * wh.abs() + O.TINY[dtype], "h")
    if f is not None:
        r2 = 1 / torch.sqrt((f.double() ** 2).mean(-1) + eps)
        within(stats[0], r2, rel * r2, "r_post")
    within(stats[1], r1[:, 0], 3 * rel * r1[:, 0], "r_pre")


def _norm_grads(x, f, gate, w2, w1, gy, gh, a, eps, per):
    """By differentiating the 64-bit form, and the magnitudes of the terms."""
    leaves = [None if t is None else t.double().requires_grad_() for t in (x, f, gate, w2, w1)]
    y, h = O.norm_gate(*leaves, a, eps, per)
    have = [t for t in leaves if t is not None]
    grads = torch.autograd.grad([y, h], have, [torch.zeros_like(y) if gy is None else gy.double(), gh.double()],
                                allow_unused=True)
    it = iter(grads)
    return [None if t is None else next(it) for t in leaves], y.detach(), h.detach()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,c,per", NORM_SIZES)
@pytest.mark.parametrize("parts,with_gy", [("fgw", True), ("fgw", False), ("f", True), ("w", True)])
def test_norm_gate_backward(dtype, rows, c, per, parts, with_gy):
    g = gen(c + 1)
    x, f, gate, w2, w1 = _norm_case(g, rows, c, per, dtype, parts)
    gy, gh = (rand(g, rows, c, dtype=dtype) if with_gy else None), rand(g, rows, c, dtype=dtype)
    eps, a = 1e-3, 0.6
    _, _, stats = T.norm_gate(x, f, gate, w2, w1, a, eps, per)
    got = T.norm_gate_backward(gy, gh, x, f, gate, w2, w1, stats, a, per)
    want, y, _ = _norm_grads(x, f, gate, w2, w1, gy, gh, a, eps, per)
    # magnitudes along the formula, in fp32 with sums of c terms
    rel = 4 * (c / 64 + 24) * O.E
    gyd, ghd = (torch.zeros_like(y) if gy is None else gy.double()), gh.double()
    one = torch.ones(c, dtype=torch.double, device=DEV)
    w1d, w2d = (one if w1 is None else w1.double()), (one if w2 is None else w2.double())
    r1 = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
    ymag = (x.double().abs() + (y - x.double()).abs())
    yh, d1 = ymag * r1, (ghd * w1d).abs()
    tmag = gyd.abs() + r1 * (d1 + yh * (d1 * yh).mean(-1, keepdim=True))
    within(got[0], want[0], O.U[dtype] * want[0].abs() + rel * tmag + O.TINY[dtype], "gx")
    if f is not None:
        gd = torch.ones_like(y) if gate is None else gate.double().abs().repeat_interleave(per, 0)[:rows]
        r2 = 1 / torch.sqrt((f.double() ** 2).mean(-1, keepdim=True) + eps)
        fh = f.double().abs() * r2
        d2 = a * tmag * gd * w2d.abs()
        fmag = r2 * (d2 + fh * (d2 * fh).mean(-1, keepdim=True))
        within(got[1], want[1], O.U[dtype] * want[1].abs() + 2 * rel * fmag + O.TINY[dtype], "gf")
        along = a * tmag * fh
        chain = rel + (rows + 64) * O.E  # at most every row in one chain
        if gate is not None:
            gates = torch.stack([s.sum(0) for s in along.split(per)])
            within(got[2], want[2], chain * gates * w2d.abs(), "ggate")
        if w2 is not None:
            within(got[3], want[3], chain * (along * gd).sum(0), "gw_post")
    if w1 is not None:
        within(got[4], want[4], (rel + (rows + 64) * O.E) * (ghd.abs() * yh).sum(0), "gw_pre")
    # the fixed order of the sums: the same bits again
    again = T.norm_gate_backward(gy, gh, x, f, gate, w2, w1, stats, a, per)
    assert all((p is None and r is None) or torch.equal(p, r) for p, r in zip(got, again))


def test_norm_gate_gradient_against_differences():
    g = gen(8)
    rows, c, per, a, eps = 12, 40, 5, 0.7, 1e-3
    args = list(_norm_case(g, rows, c, per, F32, "fgw"))
    gy, gh = rand(g, rows, c), rand(g, rows, c)
    live = [t.clone().requires_grad_() for t in args]
    y, h = T.NormGate.apply(*live, a, eps, per)
    torch.autograd.backward([y, h], [gy, gh])
    for n, t in enumerate(live):
        d = rand(g, *t.shape).double()

        def value(s):
            moved = [u.double() + (s * d if m == n else 0) for m, u in enumerate(args)]
            oy, oh = O.norm_gate(*moved, a, eps, per)
            return (oy * gy + oh * gh).sum()

        step = 1e-4
        slope = ((value(step) - value(-step)) / (2 * step)).item()
        assert abs((t.grad.double() * d).sum().item() - slope) <= 2e-5 * (t.grad.double() * d).abs().sum().item() + 1e-6


def test_norm_gate_in_place_and_misaligned():
    g = gen(9)
    x, f, gate, w2, w1 = _norm_case(g, 21, 256, 8, BF16, "fgw")
    y, h, stats = T.norm_gate(x, f, gate, w2, w1, 0.5, 1e-6, 8)
    y2, f2, s2 = x.clone(), f.clone(), torch.empty_like(stats)
    L.gs_norm_gate_fwd(y2, f2, gate, w2, w1, y2, f2, s2, 8, 0.5, 1e-6)  # y over x, h over f
    assert torch.equal(y2, y) and torch.equal(f2, h) and torch.equal(s2, stats)
    off = torch.empty(21 * 256 + 1, dtype=BF16, device=DEV)[1:].view(21, 256)  # rows off 16 bytes
    off.copy_(x)
    y3, h3, _ = T.norm_gate(off, f, gate, w2, w1, 0.5, 1e-6, 8)
    u = 2 * O.U[BF16]
    within(y3, y.double(), u * y.double().abs(), "misaligned y")
    within(h3, h.double(), u * h.double().abs(), "misaligned h")


# ---- choice of key blocks -------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("b,n,h,d,cut", [(1, 1, 1, 8, None), (2, 63, 3, 64, None), (2, 300, 2, 128, (300, 77)),
                                         (2, 129, 1, 256, (0, 128)), (1, 64, 2, 40, None), (1, 1000, 1, 24, (999,))])
def test_block_summary(dtype, b, n, h, d, cut):
    g = gen(n)
    k = 3 * rand(g, b, n, h, d, dtype=dtype)
    k[:, ::7] *= 60  # some saturate
    k[0, 0, 0, 0] = float("inf")
    length = None if cut is None else torch.tensor(cut, dtype=torch.int32, device=DEV)
    if cut:
        k[torch.arange(n, device=DEV)[None] >= length[:, None]] = float("nan")
    eight, scale = T.block_summary(k, length)
    we, ws = O.summary(k, 64, length)
    assert torch.equal(eight.long(), we) and torch.equal(scale.double(), ws)
    # a growing cache: only the last blocks again, into a transposed layout
    late = max(0, (n + 63) // 64 - 1)
    out = (torch.full((b, (n + 63) // 64, h, d), 99, dtype=torch.int8, device=DEV).transpose(1, 2),
           torch.full((b, (n + 63) // 64, h), 9.0, device=DEV).transpose(1, 2))
    T.block_summary(k, length, out, late)
    assert torch.equal(out[0][:, :, late:].long(), we[:, :, late:]) and torch.equal(out[1][:, :, late:].double(), ws[:, :, late:])
    assert (out[0][:, :, :late] == 99).all() and (out[1][:, :, :late] == 9).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("b,lq,lk,hq,hk,d,top,cut", [
    (1, 1, 1, 1, 1, 64, 1, None), (1, 1, 5000, 4, 2, 128, 9, None), (2, 130, 700, 6, 3, 64, 4, (700, 300)),
    (1, 257, 257, 2, 1, 128, 3, None), (2, 200, 100, 2, 2, 40, 2, (100, 0)), (1, 5, 64, 1, 1, 8, 40, None),
    (1, 3, 40000, 1, 1, 64, 100, None), (2, 300, 300, 2, 2, 256, 1, (130, 65))])
def test_select_blocks(causal, b, lq, lk, hq, hk, d, top, cut):
    g = gen(lk)
    q, k = rand(g, b, lq, hq, d, dtype=BF16), rand(g, b, lk, hk, d, dtype=BF16)
    length = None if cut is None else torch.tensor(cut, dtype=torch.int32, device=DEV)
    sums = T.block_summary(k, length)
    got = T.select_blocks(q, sums, lk, top, length, causal)
    assert torch.equal(got.cpu(), O.select(q, O.summary(k, 64, length), lk, top, length, causal))


def test_select_ties_go_to_the_lowest_block():
    g = gen(2)
    q = rand(g, 1, 128, 1, 64, dtype=F16)
    k = rand(g, 1, 64, 1, 64, dtype=F16).repeat(1, 50, 1, 1)  # fifty equal blocks
    k[:, 64 * 30: 64 * 31] = 0  # and one that scores zero
    sums = T.block_summary(k)
    got = T.select_blocks(q, sums, 3200, 12)[0, 0, 0].tolist()
    want = O.select(q, O.summary(k, 64), 3200, 12)[0, 0, 0].tolist()
    assert got == want
    assert got in (list(range(12)), [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 30])
    zero = torch.zeros_like(q)
    assert T.select_blocks(zero, sums, 3200, 12)[0, 0, 0].tolist() == list(range(12))


def test_select_strided_summaries_and_the_longest_cache():
    g = gen(4)
    q, k = rand(g, 1, 2, 2, 64, dtype=BF16), rand(g, 1, 900, 2, 64, dtype=BF16)
    sums = T.block_summary(k)
    want = T.select_blocks(q, sums, 900, 5)
    turned = tuple(s.transpose(1, 2).contiguous().transpose(1, 2) for s in sums)
    assert torch.equal(T.select_blocks(q, turned, 900, 5), want)
    odd = torch.empty(sums[0].numel() + 3, dtype=torch.int8, device=DEV)[3:].view(sums[0].shape)
    odd.copy_(sums[0])
    assert torch.equal(T.select_blocks(q, (odd, sums[1]), 900, 5), want)
    n = L.GS_MAX_SELECT_TOKENS  # 32768 blocks: the scores fill 128 KiB of LDS
    eight = torch.randint(-127, 128, (1, 1, n // 64, 8), generator=g, device=DEV, dtype=torch.int8)
    scale = torch.ones(1, 1, n // 64, device=DEV)
    q = rand(g, 1, 1, 1, 8)
    got = T.select_blocks(q, (eight, scale), n, 50)
    assert torch.equal(got.cpu(), O.select(q, (eight.long(), scale.double()), n, 50))


# ---- attention ------------------------------------------------------------------
def random_lists(g, b, h, groups, blocks, top, share=0.8):
    """Random ascending lists with -1 after them, some empty."""
    out = torch.full((b, h, groups, top), -1, dtype=torch.int32)
    for i in range(b):
        for j in range(h):
            for m in range(groups):
                n = min(top, blocks, int(torch.randint(0, top + 1, (1,), generator=g, device=DEV)) if (i + j + m) % 3 else top)
                ids = torch.randperm(blocks, generator=g, device=DEV)[:n].sort().values
                out[i, j, m, :n] = ids.int().cpu()
    return out.to(DEV)


ATTENTION = [
    # b, lq, lk, hq, hk, d, top, kv_len
    (1, 1, 1, 1, 1, 64, 1, None),
    (1, 1, 1000, 2, 1, 128, 16, None),          # one token, split over its list
    (2, 5, 300, 3, 3, 64, 4, (300, 111)),
    (2, 130, 200, 4, 2, 128, 3, (200, 64)),
    (1, 384, 384, 2, 1, 64, 5, None),
    (2, 100, 65, 2, 2, 128, 2, (65, 0)),        # a sequence of no keys; more queries than keys
    (1, 257, 900, 6, 1, 64, 9, None),
    (1, 33, 129, 1, 1, 128, 8, (127,)),         # lists longer than the blocks
]


def check_attention(q, k, v, lists, gout, length, causal, scale=None, backward=True):
    s = q.shape[3] ** -0.5 if scale is None else scale
    want, bound = O.attention(q, k, v, lists, s, length, causal, gout if backward else None)
    out, lse = T.block_attention(q, k, v, lists, scale, length, causal)
    within(out, want["out"], bound["out"], "out")
    within(lse, want["lse"], bound["lse"], "lse")
    if backward:
        grads = T.block_attention_backward(gout, q, k, v, out, lse, lists, scale, length, causal)
        for name, x in zip(("gq", "gk", "gv"), grads):
            within(x, want[name], bound[name], name)
        again = T.block_attention_backward(gout, q, k, v, out, lse, lists, scale, length, causal)
        assert all(torch.equal(x, y) for x, y in zip(grads, again))
    return out, lse


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("b,lq,lk,hq,hk,d,top,cut", ATTENTION)
def test_attention(dtype, causal, b, lq, lk, hq, hk, d, top, cut):
    g = gen(lq + lk)
    q, gout = (rand(g, b, lq, hq, d, dtype=dtype) for _ in range(2))
    k, v = (rand(g, b, lk, hk, d, dtype=dtype) for _ in range(2))
    length = None if cut is None else torch.tensor(cut, dtype=torch.int32, device=DEV)
    if cut:  # anything may stand past a sequence's end
        past = torch.arange(lk, device=DEV)[None] >= length[:, None]
        k[past], v[past] = float("nan"), float("inf")
    lists = random_lists(g, b, hq, (lq + 127) // 128, (lk + 63) // 64, top)
    check_attention(q, k, v, lists, gout, length, causal)


@pytest.mark.parametrize("d,lq,heads", [(128, 1100, 60), (64, 1100, 60)])
def test_attention_many_groups(d, lq, heads):
    """Enough groups for the kernel of full groups, with a short last one."""
    g = gen(d)
    q, gout = (rand(g, 1, lq, heads, d, dtype=BF16) for _ in range(2))
    k, v = (rand(g, 1, lq, 4, d, dtype=BF16) for _ in range(2))
    lists = T.select_blocks(q, T.block_summary(k), lq, 6, None, True)
    check_attention(q, k, v, lists, gout, None, True)
    k[0, 700:], v[0, 700:] = float("nan"), float("nan")
    length = torch.tensor([700], dtype=torch.int32, device=DEV)
    lists = random_lists(g, 1, heads, 9, 18, 7)
    check_attention(q, k, v, lists, gout, length, True)
    check_attention(q, k, v, lists, gout, length, False)


def test_attention_few_and_many_agree():
    """The same sequence through either kernel: full groups when there are many
    heads, split lists when there are few."""
    g = gen(12)
    q, k, v = rand(g, 1, 300, 200, 64, dtype=F16), rand(g, 1, 300, 200, 64, dtype=F16), rand(g, 1, 300, 200, 64, dtype=F16)
    lists = random_lists(g, 1, 200, 3, 5, 4)
    out, lse = T.block_attention(q, k, v, lists)
    for h in (0, 199):
        one = slice(h, h + 1)
        o, e = T.block_attention(q[:, :, one], k[:, :, one], v[:, :, one], lists[:, one].contiguous())
        want, bound = O.attention(q[:, :, one], k[:, :, one], v[:, :, one], lists[:, one], 0.125)
        within(o, want["out"], bound["out"], "few")
        within(out[:, :, one], want["out"], bound["out"], "many")
        within(e, want["lse"], bound["lse"], "few lse")
        within(lse[:, one], want["lse"], bound["lse"], "many lse")


def test_attention_large_scores_and_scales():
    """Scores of several hundred, equal scores, and a value range near the type's largest."""
    g = gen(6)
    for dtype, big in ((F16, 3e4), (BF16, 1e30)):
        q, k, v = (rand(g, 1, 140, 2, 64, dtype=dtype) for _ in range(3))
        gout = rand(g, 1, 140, 2, 64, dtype=dtype)
        lists = random_lists(g, 1, 2, 2, 3, 3)
        check_attention(30 * q, 3 * k, v, lists, gout, None, True, scale=0.5, backward=False)
        check_attention(torch.zeros_like(q), k, v, lists, gout, None, False)
        check_attention(q, k, (v.float() * (big / v.abs().max().float())).to(dtype), lists, gout, None, False, backward=False)


def test_attention_malformed_lists_stay_inside():
    """Repeated, descending, negative and too large entries are skipped in both
    directions."""
    g = gen(7)
    q, gout = rand(g, 1, 250, 2, 64, dtype=BF16), rand(g, 1, 250, 2, 64, dtype=BF16)
    k, v = rand(g, 1, 310, 2, 64, dtype=BF16), rand(g, 1, 310, 2, 64, dtype=BF16)
    big = 2 ** 31 - 1
    rows = [[0, 0, 2, 2, 4], [3, 1, -1, -5, -1], [1, 5, 6, big, -7], [-1, -1, -1, -1, -1]]
    lists = torch.tensor(rows, dtype=torch.int32, device=DEV).view(1, 2, 2, 5)
    check_attention(q, k, v, lists, gout, None, False)
    check_attention(q, k, v, lists, gout, None, True)


def test_attention_strides_streams_and_autograd():
    g = gen(10)
    b, n, h, d = 2, 200, 3, 64
    packed = rand(g, b, n, 3, h, d, dtype=BF16)
    q, k, v = packed.unbind(2)
    gout = rand(g, b, h, n, d, dtype=BF16).transpose(1, 2)
    lists = random_lists(g, b, h, 2, 4, 3)
    out, lse = check_attention(q, k, v, lists, gout, None, True)
    # rows off 16 bytes are copied
    odd = torch.empty(packed.numel() + 1, dtype=BF16, device=DEV)[1:].view(packed.shape)
    odd.copy_(packed)
    o2, l2 = T.block_attention(*odd.unbind(2), lists, None, None, True)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    # heads first, on another stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hf = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v)]
        o3, l3 = T.block_attention(*hf, lists, None, None, True)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o3, out) and torch.equal(l3, lse)
    live = packed.clone().requires_grad_()
    ql, kl, vl = live.unbind(2)
    T.BlockAttention.apply(ql, kl, vl, lists, None, None, True).backward(gout)
    grads = T.block_attention_backward(gout, q, k, v, out, lse, lists, None, None, True)
    assert torch.equal(live.grad, torch.stack(grads, 2))


def test_attention_gradient_against_differences():
    """The gradient along a direction, against differences of the 64-bit form."""
    g = gen(13)
    b, n, h, d = 1, 150, 2, 64
    x = [rand(g, b, n, h, d, dtype=F16) for _ in range(3)]
    gout = rand(g, b, n, h, d, dtype=F16)
    lists = random_lists(g, b, h, 2, 3, 2)
    out, lse = T.block_attention(*x, lists, None, None, True)
    grads = T.block_attention_backward(gout, *x, out, lse, lists, None, None, True)
    bound = O.attention(*x, lists, 0.125, None, True, gout)[1]
    for m, name in enumerate(("gq", "gk", "gv")):
        way, step = rand(g, b, n, h, d).double(), 1e-4

        def value(s):
            moved = [t.double() + (s * way if i == m else 0) for i, t in enumerate(x)]
            o = torch.zeros(b, n, h, d, dtype=torch.double, device=DEV)
            for j in range(h):
                on = O.listed(lists[0, j], 3).repeat_interleave(128, 0)[:n].repeat_interleave(64, 1)[:, :n]
                on = on & torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
                s_ = (moved[0][0, :, j] @ moved[1][0, :, j].T.contiguous() * 0.125).masked_fill(~on, -math.inf)
                o[0, :, j] = torch.nan_to_num(torch.softmax(s_, 1)) @ moved[2][0, :, j]
            return (o * gout.double()).sum()

        slope = ((value(step) - value(-step)) / (2 * step)).item()
        along = (grads[m].double() * way).sum().item()
        assert abs(along - slope) <= (bound[name] * way.abs()).sum().item() + 1e-6


def test_offsets_past_32_bits():
    """One head of a wide cache of 300,000 tokens: elements past 2^31."""
    g = gen(14)
    tokens, wide, d = 300_000, 8192, 64
    cache = [torch.empty(tokens, wide, dtype=BF16, device=DEV) for _ in range(2)]
    blocks = [0, 2000, (tokens + 63) // 64 - 1]
    rows = torch.cat([torch.arange(m * 64, min(tokens, m * 64 + 64), device=DEV) for m in blocks])
    small = [rand(g, 1, rows.numel(), 1, d, dtype=BF16) for _ in range(2)]
    views = []
    for c, s in zip(cache, small):
        c[rows, wide - d:] = s[0, :, 0]
        views.append(c[None, :, None, wide - d:])
    q = rand(g, 1, 3, 1, d, dtype=BF16)
    lists = torch.tensor(blocks, dtype=torch.int32, device=DEV).view(1, 1, 1, 3)
    out, lse = T.block_attention(q, *views, lists)
    near = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV).view(1, 1, 1, 3)
    o2, l2 = T.block_attention(q, *small, near)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    gout = rand(g, 1, 3, 1, d, dtype=BF16)
    grads = T.block_attention_backward(gout, q, *views, out, lse, lists)
    near_grads = T.block_attention_backward(gout, q, *small, o2, l2, near)
    assert torch.equal(grads[0], near_grads[0])
    for x, y in zip(grads[1:], near_grads[1:]):
        assert torch.equal(x[0, rows], y[0])
        assert int((x != 0).any(-1).sum()) <= rows.numel()
    eight, _ = T.block_summary(views[0])
    assert torch.equal(eight[0, 0, blocks], T.block_summary(small[0])[0][0, 0])


def test_empty_sizes():
    q = torch.zeros(1, 0, 2, 64, dtype=BF16, device=DEV)
    k = torch.ones(1, 70, 1, 64, dtype=BF16, device=DEV)
    lists = torch.empty(1, 2, 0, 3, dtype=torch.int32, device=DEV)
    out, lse = T.block_attention(q, k, k, lists)
    assert out.shape == q.shape and lse.shape == (1, 2, 0)
    gq, gk, gv = T.block_attention_backward(q, q, k, k, out, lse, lists)
    assert not gk.any() and not gv.any()
    q = torch.ones(1, 9, 2, 64, dtype=BF16, device=DEV)
    none = torch.zeros(1, 0, 1, 64, dtype=BF16, device=DEV)
    lists = T.select_blocks(q, T.block_summary(none), 0, 3)
    assert (lists == -1).all()
    out, lse = T.block_attention(q, none, none, lists)
    assert not out.any() and (lse == -math.inf).all()
    gq, gk, gv = T.block_attention_backward(q, q, none, none, out, lse, lists)
    assert not gq.any() and gk.shape == none.shape
    x = torch.zeros(0, 8, device=DEV)
    w = torch.ones(8, device=DEV)
    gate = torch.ones(0, 8, device=DEV)
    y, h, stats = T.norm_gate(x, x, gate, w, w, rows_per_gate=4)
    grads = T.norm_gate_backward(x, x, x, x, gate, w, w, stats, rows_per_gate=4)
    assert not grads[3].any() and not grads[4].any()
    pos = torch.zeros(1, 0, 3, dtype=torch.int32, device=DEV)
    r = torch.zeros(2, 0, 1, 8, device=DEV)
    assert T.rope_axes(r, None, pos, torch.ones(4, device=DEV), (1, 1, 1))[0].shape == r.shape
