"""Layer norm, the gated feed-forward block and 4-bit linear layers from their
definitions in 64 bits, for the GPU tests, with what their error bounds are made
of: the sums of magnitudes that roundings are relative to."""

import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half an ulp, relative
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the least subnormal
E = 2.0 ** -24


def within(got, want, bound, what):
    """Every element within its bound; what is not finite, the same."""
    got, fine = got.double(), torch.isfinite(want)
    assert got.shape == want.shape, what
    assert torch.equal(torch.isfinite(got), fine), f"{what}: other elements are finite"
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: other elements are NaN"
    over = ((got - want).abs() - bound)[fine]
    assert over.numel() == 0 or over.max() <= 0, f"{what}: {over.max().item():.3e} over the bound"


def layer_norm(x, w, b, eps):
    x = x.double()
    x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())


def layer_norm_gradients(gy, x, w, eps):
    """gx, gw, gb and the magnitudes that their roundings are relative to."""
    x, gy = x.double(), gy.double()
    w = torch.ones(x.shape[1], dtype=torch.double, device=x.device) if w is None else w.double()
    x0 = x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((x0 * x0).mean(-1, keepdim=True) + eps)
    xh, d = x0 * r, gy * w
    gx = r * (d - d.mean(-1, keepdim=True) - xh * (d * xh).mean(-1, keepdim=True))
    # xh is off by roundings of the mean of x too
    mag = xh.abs() + r * x.abs().mean(-1, keepdim=True)
    d = d.abs()
    return ((gx, r * (d + d.mean(-1, keepdim=True) + mag * (d * mag).mean(-1, keepdim=True))),
            ((gy * xh).sum(0), (gy.abs() * mag).sum(0)), (gy.sum(0), gy.abs().sum(0)))


def activation(act, g):
    """(value, derivative) of the gate, 64 bits."""
    if act == "silu":
        t = torch.sigmoid(g)
        return g * t, t * (1 + g * (1 - t))
    f = 0.5 * torch.special.erfc(-g / math.sqrt(2))
    return g * f, f + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def gated_ff(x, w_gate, w_up, w_down, act, gy=None):
    """[y, gx, gw_gate, gw_up, gw_down], or y alone, with bounds: first order in
    the roundings, sums of n products n + 16 roundings at most."""
    kind = x.dtype
    u8, tiny = U[kind], TINY[kind]
    x, w_gate, w_up, w_down = (t.double() for t in (x, w_gate, w_up, w_down))
    (rows, c), f, co = x.shape, w_gate.shape[0], w_down.shape[0]
    chain = lambda n: (n + 16) * E  # noqa: E731
    g, u = x @ w_gate.T, x @ w_up.T
    dg, du = (chain(c) * (x.abs() @ w.abs().T) for w in (w_gate, w_up))
    a, da = activation(act, g)
    # slopes of act and act' are below 1.13 and 0.8; the function itself: 16 roundings and 1.5e-7 of the error function
    off = (16 * E + 1.5e-7) * g.abs()
    off_d = (16 * E + 1.5e-7) * (1 + g.abs())
    h = a * u
    dh = (1.13 * dg + off) * u.abs() + a.abs() * du + u8 * h.abs() + tiny
    y = h @ w_down.T
    dy = dh @ w_down.abs().T + chain(f) * (h.abs() @ w_down.abs().T) + u8 * y.abs() + tiny
    if gy is None:
        return [(y, 1.01 * dy)]
    gy = gy.double()
    # the backward pass's g and u are rounded to 12 or 16 significant bits
    cut = {torch.float16: 2.0 ** -16, torch.bfloat16: 2.0 ** -12}[kind]
    dg, du = dg + cut * g.abs(), du + cut * u.abs()
    gh, dgh = gy @ w_down, chain(co) * (gy.abs() @ w_down.abs())
    gg, gu = gh * u * da, gh * a
    dgg = dgh * (u * da).abs() + gh.abs() * (du * da.abs() + u.abs() * (0.8 * dg + off_d)) + u8 * gg.abs() + tiny
    dgu = dgh * a.abs() + gh.abs() * (1.13 * dg + off) + u8 * gu.abs() + tiny
    gx = gg @ w_gate + gu @ w_up
    dgx = dgg @ w_gate.abs() + dgu @ w_up.abs() + chain(2 * f) * (gg.abs() @ w_gate.abs() + gu.abs() @ w_up.abs())
    out = [(y, dy), (gx, dgx + u8 * gx.abs() + tiny)]
    for p, dp in ((gg, dgg), (gu, dgu)):
        w = p.T @ x
        out.append((w, dp.T @ x.abs() + chain(rows) * (p.abs().T @ x.abs()) + u8 * w.abs() + tiny))
    w = gy.T @ h
    out.append((w, gy.abs().T @ dh + chain(rows) * (gy.abs().T @ h.abs()) + u8 * w.abs() + tiny))
    return [(v, 1.01 * d) for v, d in out]


GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def quantise4(x):
    """(codes [rows, channels], e [rows, channels / 32], values in 64 bits)."""
    rows, c = x.shape
    v = x.double().view(rows, c // 32, 32)
    top = v.abs().amax(-1)
    fine = torch.isfinite(top) & ~torch.isnan(v).any(-1)
    # the exponent by comparison with powers of two, not by a logarithm
    e = torch.zeros(rows, c // 32, dtype=torch.long, device=x.device)
    for p in range(-124, 128):  # floor(log2 top) - 2 + 127 where that is over 0
        e += (top >= 2.0 ** p).long() * fine
    power = torch.exp2(e.double() - 127)
    m = torch.where(fine[..., None], v.abs() / power[..., None], 0.0)
    grid = torch.tensor(GRID, dtype=torch.double, device=x.device)
    d = (m[..., None] - grid).abs()
    near = d == d.amin(-1, keepdim=True)
    # of two the even code
    order = torch.tensor([0, 8, 1, 9, 2, 10, 3, 11], device=x.device)
    code = torch.where(near, order, 99).argmin(-1)
    value = torch.where(fine[..., None], torch.copysign(grid[code], v) * power[..., None], float("nan"))
    code = code + 8 * torch.signbit(v).long()
    return code.view(rows, c), torch.where(fine, e, 255), value.view(rows, c), fine


def unpack4(codes, scales, channels):
    """The values of a packed pair, in 64 bits."""
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(1).long()
    grid = torch.tensor([*GRID, *(-g for g in GRID)], dtype=torch.double, device=codes.device)
    e = scales[:, : channels // 32].long()
    power = torch.where(e == 255, float("nan"), torch.exp2(e.double() - 127))
    return grid[both] * power.repeat_interleave(32, 1)
