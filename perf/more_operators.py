"""The dense half of a layer of tile tokens as a user calls it, and its plain forms.

A token is a 16x16 tile of a view (the rasterizer's tile), so the sizes below
are those of the repository's images: 256x256 is 256 tokens, 1280x720 is 3600,
four 1920x1080 views are 32640. A tile's pixels are 768 values, the predictor's
stream has 256 channels and a hidden layer four times as wide.

Three operators: layer norm, forward and backward; the gated feed-forward block
(two projections, the activation of one times the other, the projection back),
forward and backward; and linear layers in microscaled 4-bit floating point
(blocks of 32 values with a power of two each) for serving.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
SIZE = 32  # values that share a scale
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes of 4 bits


# ---- cases --------------------------------------------------------------------
def listed():
    return [
        # the pixels of one small image's tiles before the embedding, when serving: latency counts
        dict(name="layer-256sq", op="layer", rows=256, channels=768, type="bf16", affine=True, train=False),
        # a training step over two 720p views in fp32 at a channel count that no vector width divides, without weights
        dict(name="layer-720p-f32", op="layer", rows=7200, channels=1027, type="f32", affine=False, train=True),
        # a training step over four 1080p views
        dict(name="layer-4x1080p", op="layer", rows=32640, channels=2048, type="bf16", affine=True, train=True),
        # one new token through a wide layer: the weights are read once
        dict(name="gated-one", op="gated", rows=1, channels=2048, hidden=8192, act="silu", type="bf16", train=False),
        # a few tokens at odd sizes in a training step, fp16
        dict(name="gated-few-f16", op="gated", rows=45, channels=520, hidden=1368, act="gelu", type="f16", train=True),
        # the predictor's own layer over one 256x256 image, a training step
        dict(name="gated-256sq", op="gated", rows=256, channels=256, hidden=1024, act="gelu", type="bf16", train=True),
        # one 720p view when serving, fp16
        dict(name="gated-720p-f16", op="gated", rows=3600, channels=1024, hidden=4096, act="silu", type="f16", train=False),
        # a training step over four 1080p views
        dict(name="gated-4x1080p", op="gated", rows=32640, channels=2048, hidden=8192, act="silu", type="bf16", train=True),
        # activations to 4 bits and back, four 1080p views
        dict(name="pack-4x1080p", op="pack", rows=32640, channels=2048, type="bf16"),
        # one new token against 4-bit weights: they are read once
        dict(name="four-one", op="four", rows=1, channels=2048, out=8192, type="bf16"),
        # a 720p view at channel counts off every tile, fp16
        dict(name="four-720p-f16", op="four", rows=3600, channels=1056, out=1000, type="f16"),
        # four 1080p views, the widest layer
        dict(name="four-4x1080p", op="four", rows=32640, channels=2048, out=8192, type="bf16"),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["layer", "gated", "gated", "pack", "four"])
    if op == "layer":
        channels = _log(rng, 32, 4096)
        channels = channels - channels % 8 if rng.random() < 0.5 else channels
        return dict(op=op, rows=_log(rng, 1, min(32640, 32640 * 2048 // channels)), channels=channels,
                    type=rng.choice(["f32", "f16", "bf16"]), affine=rng.random() < 0.7, train=rng.random() < 0.6)
    if op == "pack":
        channels = SIZE * _log(rng, 1, 128)
        return dict(op=op, rows=_log(rng, 1, min(32640, 32640 * 2048 // channels)), channels=channels,
                    type=rng.choice(["f32", "f16", "bf16"]))
    few = rng.random() < 0.3
    if op == "four":
        return dict(op=op, rows=rng.randint(1, 16) if few else _log(rng, 17, 16320), channels=SIZE * _log(rng, 2, 128),
                    out=_log(rng, 64, 8192), type=rng.choice(["f32", "f16", "bf16"]))
    return dict(op=op, rows=rng.randint(1, 16) if few else _log(rng, 17, 16320), channels=8 * _log(rng, 8, 256),
                hidden=8 * _log(rng, 16, 1024), act=rng.choice(["silu", "gelu"]), type=rng.choice(["f16", "bf16"]),
                train=not few and rng.random() < 0.7)


# ---- inputs -------------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _tokens(gen, rows, channels):
    """A normed stream: unit variance, a few channels far larger than the rest."""
    loud = 1.0 + 7.0 * (torch.rand(channels, generator=gen, device="cuda") < 0.01).float()
    return _normal(gen, rows, channels) * loud


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    state = dict(case)
    kind, rows, c = TYPES[case["type"]], case["rows"], case["channels"]
    if case["op"] == "layer":
        # pixels and residual streams are off zero
        state["x"] = (1.5 * _normal(gen, rows, c) + 0.8 + 0.5 * _normal(gen, rows, 1)).to(kind)
        state["w"] = 1.0 + 0.2 * _normal(gen, c) if case["affine"] else None
        state["b"] = 0.1 * _normal(gen, c) if case["affine"] else None
        state["gy"] = _normal(gen, rows, c).to(kind)
        state["eps"] = 1e-5
    elif case["op"] == "gated":
        f = case["hidden"]
        state["x"] = _tokens(gen, rows, c).to(kind)
        state["w_gate"] = (_normal(gen, f, c) / math.sqrt(c)).to(kind)
        state["w_up"] = (_normal(gen, f, c) / math.sqrt(c)).to(kind)
        state["w_down"] = (_normal(gen, c, f) / math.sqrt(f)).to(kind)
        state["gy"] = _normal(gen, rows, c).to(kind)
    else:
        state["x"] = _tokens(gen, rows, c).to(kind)
        if case["op"] == "four":
            # a serving program holds its weights in 4 bits
            state["weights"] = _to_four(_normal(gen, case["out"], c) / math.sqrt(c))
    return state


def _to_four(x):
    """uint8 codes [rows, channels / 2] (value 2 i in the low half of byte i) and
    uint8 scales [rows, channels / 32, filled up to a multiple of 4]."""
    rows, c = x.shape
    block = x.float().view(rows, c // SIZE, SIZE)
    power = _power(block)
    value = _rounded(block, power)
    grid = torch.tensor(GRID, device="cuda")
    code = torch.bucketize(value.abs(), grid) + 8 * (value < 0)
    code = code.view(rows, c // 2, 2).to(torch.uint8)
    byte = (power + 127).to(torch.uint8)[..., 0]
    return code[..., 0] + 16 * code[..., 1], torch.nn.functional.pad(byte, (0, -(c // SIZE) % 4))


# ---- plain forms --------------------------------------------------------------
def _layer_plain(s):
    x, kind = s["x"].float(), s["x"].dtype
    x0 = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x0 * x0).mean(-1, keepdim=True) + s["eps"])
    xh = x0 * r
    w = 1.0 if s["w"] is None else s["w"]
    y = xh * w + (0.0 if s["b"] is None else s["b"])
    if not s["train"]:
        return [y.to(kind)]
    gy = s["gy"].float()
    d = gy * w
    gx = r * (d - d.mean(-1, keepdim=True) - xh * (d * xh).mean(-1, keepdim=True))
    return [y.to(kind), gx.to(kind)] + ([(gy * xh).sum(0), gy.sum(0)] if s["affine"] else [])


def _act_plain(act, g):
    """The activation and its derivative."""
    if act == "silu":
        t = 1.0 / (1.0 + torch.exp(-g))
        return g * t, t * (1.0 + g * (1.0 - t))
    t = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return g * t, t + g * torch.exp(-0.5 * g * g) * (0.5 / math.pi) ** 0.5


def _gated_plain(s):
    kind = s["x"].dtype
    x, w_gate, w_up, w_down = (s[n].float() for n in ("x", "w_gate", "w_up", "w_down"))
    g, u = x @ w_gate.t(), x @ w_up.t()
    a, da = _act_plain(s["act"], g)
    h = a * u
    y = (h @ w_down.t()).to(kind)
    if not s["train"]:
        return [y]
    gy = s["gy"].float()
    gh = gy @ w_down
    gg, gu = gh * u * da, gh * a
    return [y, (gg @ w_gate + gu @ w_up).to(kind), (gg.t() @ x).to(kind), (gu.t() @ x).to(kind), (gy.t() @ h).to(kind)]


def _power(block):
    """The exponent of each block of 32: its largest magnitude's, less that of 4."""
    largest = block.abs().amax(-1, keepdim=True)
    return torch.where(largest > 0.0, torch.frexp(largest)[1] - 3, -127).clamp_min(-127)


def _rounded(block, power):
    """To the grid of magnitudes, in steps of 1/2, 1 or 2; halves to even."""
    v = torch.ldexp(block, -power)
    m = v.abs()
    step = torch.where(m < 2.0, 0.5, torch.where(m < 4.0, 1.0, 2.0))
    return torch.copysign(((m / step).round() * step).clamp_max(6.0), v)


def _four_values(x):
    block = x.float().unflatten(1, (-1, SIZE))
    power = _power(block)
    return torch.ldexp(_rounded(block, power), power).flatten(1), (power + 127).to(torch.uint8)[..., 0]


def _from_four(codes, scales, channels):
    grid = torch.tensor([*GRID, *(-g for g in GRID)], device="cuda")
    value = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).flatten(1)
    power = scales[:, : channels // SIZE].int() - 127
    return torch.ldexp(value.unflatten(1, (-1, SIZE)), power[..., None]).flatten(1)


def _plain(s):
    if s["op"] == "layer":
        return _layer_plain(s)
    if s["op"] == "gated":
        return _gated_plain(s)
    values, scales = _four_values(s["x"])
    if s["op"] == "pack":
        return [values.to(s["x"].dtype), scales]
    return [(values @ _from_four(*s["weights"], s["channels"]).t()).to(s["x"].dtype)]


# ---- the framework's calls ----------------------------------------------------
def _framework(s):
    from gaussian_splatting_differentiable_ewa_amd import tokens as T

    if s["op"] == "layer":
        y, stats = T.layer_norm(s["x"], s["w"], s["b"], eps=s["eps"])
        if not s["train"]:
            return [y]
        gx, gw, gb = T.layer_norm_backward(s["gy"], s["x"], s["w"], stats, bias=s["b"] is not None)
        return [y, gx] + ([gw, gb] if s["affine"] else [])
    if s["op"] == "gated":
        weights = s["w_gate"], s["w_up"], s["w_down"]
        if not s["train"]:
            return [T.gated_ff(s["x"], *weights, act=s["act"])]
        y, h, pre = T.gated_ff_train(s["x"], *weights, act=s["act"])
        return [y, *T.gated_ff_backward(s["gy"], s["x"], *weights, h, pre, act=s["act"])]
    if s["op"] == "pack":
        four = T.quantise4(s["x"])
        return [T.dequantise4(four, s["x"].dtype), four[1][:, : s["channels"] // SIZE]]
    return [T.linear4(s["x"], s["weights"])]


def run(state):
    return _framework(state) if own else _plain(state)


# ---- what a pass cannot do without --------------------------------------------
def work(case):
    size, rows, c = BYTES[case["type"]], case["rows"], case["channels"]
    if case["op"] == "layer":
        values, vectors = rows * c, (4 * c * (4 if case["train"] else 2) if case["affine"] else 0)
        # forward: x in, y out; backward: gy in, gx out (x read once for both)
        return {"bytes": size * values * (4 if case["train"] else 2) + vectors, "flops": values * (20 if case["train"] else 8)}
    if case["op"] == "gated":
        f = case["hidden"]
        if not case["train"]:
            return {"bytes": size * (2 * rows * c + 3 * f * c), "flops": 6 * rows * f * c}
        return {"bytes": size * (4 * rows * c + 6 * f * c), "flops": 18 * rows * f * c}
    if case["op"] == "pack":
        # x in, its values out, and the 4-bit form between them, which is the result, out
        return {"bytes": rows * c * 2 * size + rows * (c // 2 + c // SIZE), "flops": 6 * rows * c}
    n = case["out"]
    return {"bytes": size * rows * (c + n) + n * (c // 2 + c // SIZE), "flops": 2 * rows * c * n}


# ---- the definitions in 64 bits -----------------------------------------------
def _exact_layer(s):
    # the gradients by differentiating the forward formula
    x = s["x"].double().requires_grad_()
    extra = [s[n].double().requires_grad_() for n in ("w", "b")] if s["affine"] else []
    variance, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    y = (x - mean) / (variance + s["eps"]).sqrt()
    if extra:
        y = y * extra[0] + extra[1]
    if not s["train"]:
        return [y.detach()]
    return [y.detach(), *torch.autograd.grad(y, [x, *extra], s["gy"].double())]


def _exact_gated(s):
    leaves = [s[n].double().requires_grad_() for n in ("x", "w_gate", "w_up", "w_down")]
    x, w_gate, w_up, w_down = leaves
    g = x @ w_gate.T
    gate = g * torch.sigmoid(g) if s["act"] == "silu" else g * (1.0 - torch.erfc(g / 2 ** 0.5) / 2)
    y = (gate * (x @ w_up.T)) @ w_down.T
    if not s["train"]:
        return [y.detach()]
    return [y.detach(), *torch.autograd.grad(y, leaves, s["gy"].double())]


def _exact_four(x):
    """The nearest of the grid's magnitudes by distance; of two, the one with an
    even code."""
    block = x.double().unflatten(1, (-1, SIZE))
    largest = block.abs().amax(-1, keepdim=True)
    # largest magnitude / 4, rounded down to a power of two
    power = torch.where(largest > 0, torch.exp2(torch.floor(torch.log2(largest)) - 2.0), 2.0 ** -127)
    v = (block / power).abs()
    best, off = torch.zeros_like(v), v.clone()
    for i in (2, 4, 6, 1, 3, 5, 7):  # even codes first, so that they keep what is equally near
        d = (v - GRID[i]).abs()
        best, off = torch.where(d < off, GRID[i], best), torch.minimum(d, off)
    return (best * power * block.sign()).flatten(1), power[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer":
        return _exact_layer(s)
    if case["op"] == "gated":
        return _exact_gated(s)
    values, power = _exact_four(s["x"])
    if case["op"] == "pack":
        return [values, (power.log2() + 127.0).round().to(torch.uint8)]
    codes, scales = s["weights"]
    low, high = (codes % 16).long(), (codes // 16).long()
    both = torch.stack([low, high], -1).flatten(1)
    weight = torch.tensor(GRID, device="cuda", dtype=torch.double)[both % 8] * (1 - 2 * (both // 8))
    weight = weight * torch.exp2(scales.double() - 127.0).repeat_interleave(SIZE, 1)[:, : case["channels"]]
    return [values @ weight.T]
