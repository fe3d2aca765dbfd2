"""The token operators as a user calls them, and their plain forms.

A token is a 16x16 tile of a view (the rasterizer's tile), so the sizes below
are those of the repository's images: 256x256 is 256 tokens, two 250x190 views
384, 1280x720 is 3600, 3840x2160 is 32400, four 1920x1080 views 32640 and
sixteen 130560.

Four operators: rotary positions over (view, row, column); the norms after and
before a block with its gate and residual scale; the choice of key blocks by a
cheap score; the attention over the chosen blocks.
"""

import math

import torch

own = False

GROUP = 128  # consecutive queries that share a list
BLOCK = 64   # consecutive keys of a block
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---- cases --------------------------------------------------------------------
def listed():
    return [
        # the smallest image's tokens in one block of a small network: latency counts
        dict(name="rope-256sq", op="rope", batch=1, tokens=256, hq=8, hk=8, dim=64, type="bf16", pairs="8 12 12",
             interleaved=False, inverse=False),
        # the gradient's way back through the positions, two 250x190 views in fp32, fewer key heads, a part left unrotated
        dict(name="rope-ragged-back", op="rope", batch=2, tokens=384, hq=12, hk=4, dim=96, type="f32",
             pairs="8 16 16", interleaved=True, inverse=True),
        # four 1080p views, the widest heads
        dict(name="rope-4x1080p", op="rope", batch=1, tokens=32640, hq=16, hk=16, dim=128, type="bf16",
             pairs="16 24 24", interleaved=False, inverse=False),
        # one small image when serving: forward alone
        dict(name="norm-256sq", op="norm", rows=256, channels=512, per_gate=256, type="bf16", train=False),
        # a training step's norms in fp32 at a channel count that no vector width divides, one gate per 720p view
        dict(name="norm-720p-f32", op="norm", rows=7200, channels=1027, per_gate=3600, type="f32", train=True),
        # a training step's norms over four 1080p views
        dict(name="norm-4x1080p", op="norm", rows=32640, channels=2048, per_gate=8160, type="bf16", train=True),
        # one new token against the summaries of sixteen 1080p views' cache
        dict(name="select-one", op="select", batch=1, lq=1, lk=130560, hq=16, hk=4, dim=128, top=32, type="bf16",
             causal=True, ragged=False),
        # all tokens of four 1080p views among themselves, summaries made in the call
        dict(name="select-4x1080p", op="select", batch=1, lq=32640, lk=32640, hq=16, hk=16, dim=128, top=32,
             type="bf16", causal=False, ragged=False),
        # one new token's attention over its 32 blocks of that cache
        dict(name="attend-one", op="attend", batch=1, lq=1, lk=130560, hq=16, hk=4, dim=128, top=32, type="bf16",
             causal=True, ragged=False, train=False),
        # a small ragged batch in training: two pairs of 250x190 views, one pair shorter, fp16, shared key heads
        dict(name="attend-ragged", op="attend", batch=2, lq=384, lk=384, hq=12, hk=4, dim=64, top=3, type="f16",
             causal=True, ragged=True, train=True),
        # a 4K view's prompt, forward, shared key heads
        dict(name="attend-4k", op="attend", batch=1, lq=32400, lk=32400, hq=16, hk=4, dim=64, top=16, type="bf16",
             causal=True, ragged=False, train=False),
        # a training step over four 1080p views
        dict(name="attend-4x1080p", op="attend", batch=1, lq=32640, lk=32640, hq=16, hk=16, dim=128, top=32,
             type="bf16", causal=False, ragged=False, train=True),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rope", "norm", "select", "attend", "attend"])
    if op == "norm":
        channels = _log(rng, 64, 4096)
        channels = channels - channels % 8 if rng.random() < 0.5 else channels
        rows = _log(rng, 1, min(32640, 32640 * 2048 // channels))
        return dict(op=op, rows=rows, channels=channels, per_gate=max(1, rows // rng.choice([1, 2, 4])),
                    type=rng.choice(["f32", "f16", "bf16"]), train=rng.random() < 0.6)
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3]) if hk < 8 else hk * rng.choice([1, 2])
    batch = rng.choice([1, 1, 2])
    if op == "rope":
        dim = rng.choice([32, 64, 96, 128])
        half = dim // 2
        parts = rng.choice([(half, 0, 0), (0, half // 2, half // 2), (half // 4, half // 4, half // 4)])
        return dict(op=op, batch=batch, tokens=_log(rng, 1, 32640 // batch), hq=hq, hk=hk, dim=dim,
                    type=rng.choice(["f32", "f16", "bf16"]), pairs="%d %d %d" % parts, interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.5)
    dim = rng.choice([64, 128])
    one = rng.random() < 0.3
    lq = rng.randint(1, 8) if one else _log(rng, 1, 16320 // batch)
    lk = _log(rng, 64, 130560) if one else (lq if rng.random() < 0.7 else lq + _log(rng, 1, 8192))
    case = dict(op=op, batch=batch, lq=lq, lk=lk, hq=hq, hk=hk, dim=dim, top=_log(rng, 1, 48),
                type=rng.choice(["f16", "bf16"]), causal=rng.random() < 0.6, ragged=batch > 1 and rng.random() < 0.5)
    if op == "attend":
        case["train"] = not one and rng.random() < 0.7
    return case


# ---- inputs -------------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _heads(case, gen):
    """Queries and keys as after their own norms: unit variance, with clusters
    of neighbouring tokens (few of them popular) that make some blocks matter."""
    b, lq, lk, hq, hk, dim = (case[n] for n in ("batch", "lq", "lk", "hq", "hk", "dim"))
    n_blocks, clusters = (lk + BLOCK - 1) // BLOCK, 24
    centre = _normal(gen, hk, clusters, dim)
    u = torch.rand(b, n_blocks, generator=gen, device="cuda")
    of_block = (clusters * u * u).long().clamp_max(clusters - 1)
    of_key = of_block.repeat_interleave(BLOCK, 1)[:, :lk]
    of_query = of_key[:, lk - lq:] if lq <= lk else of_key.repeat(1, lq // lk + 1)[:, :lq]
    k = 0.8 * _normal(gen, b, lk, hk, dim) + 0.6 * centre[:, of_key].permute(1, 2, 0, 3)
    shared = torch.arange(hq, device="cuda") // (hq // hk)
    q = 0.8 * _normal(gen, b, lq, hq, dim) + 0.6 * centre[shared][:, of_query].permute(1, 2, 0, 3)
    return q, k


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    state = dict(case)
    kind = TYPES[case["type"]]
    if case["op"] == "rope":
        b, n, dim = case["batch"], case["tokens"], case["dim"]
        state["pairs"] = tuple(int(p) for p in case["pairs"].split())
        # one packed projection [q heads | k heads], as a model's linear layer writes it
        packed = _normal(gen, b, n, (case["hq"] + case["hk"]) * dim).to(kind)
        state["q"] = packed[..., : case["hq"] * dim].unflatten(-1, (case["hq"], dim))
        state["k"] = packed[..., case["hq"] * dim:].unflatten(-1, (case["hk"], dim))
        columns = max(1, int(math.isqrt(n)))
        first = torch.randint(0, 64, (b, 1), generator=gen, device="cuda")
        at = torch.arange(n, device="cuda")[None] + first
        state["pos"] = torch.stack([at // (columns * columns), at // columns % columns, at % columns], -1).int()
        of_axis = [torch.arange(p, device="cuda", dtype=torch.float32) / max(p, 1) for p in state["pairs"]]
        state["freq"] = torch.cat([10000.0 ** -x for x in of_axis])
        state["freq"] = torch.nn.functional.pad(state["freq"], (0, dim // 2 - state["freq"].numel()))
    elif case["op"] == "norm":
        rows, c = case["rows"], case["channels"]
        segments = (rows + case["per_gate"] - 1) // case["per_gate"]
        state["x"] = (1.5 * _normal(gen, rows, c) + 0.1).to(kind)
        state["f"] = (0.7 * _normal(gen, rows, c)).to(kind)
        state["gate"] = 0.5 + 0.3 * _normal(gen, segments, c)
        state["w_post"] = 1.0 + 0.2 * _normal(gen, c)
        state["w_pre"] = 1.0 + 0.2 * _normal(gen, c)
        state["gy"] = _normal(gen, rows, c).to(kind)
        state["gh"] = _normal(gen, rows, c).to(kind)
        state["scale"], state["eps"] = 0.7071, 1e-6
    else:
        q, k = _heads(case, gen)
        state["q"], state["k"] = q.to(kind), k.to(kind)
        b, lk = case["batch"], case["lk"]
        state["length"] = None
        if case["ragged"]:
            cut = torch.randint(0, lk // 2 + 1, (b,), generator=gen, device="cuda")
            cut[0] = 0
            state["length"] = (lk - cut).int()
            # what a cache holds past a sequence's end is anything
            past = torch.arange(lk, device="cuda")[None] >= state["length"][:, None]
            state["k"][past] = float("nan")
        if case["op"] == "select":
            # a decoding program keeps the summaries of its cache; a prompt makes them in the call
            state["summary"] = _summaries(state["k"], state["length"], BLOCK) if case["lq"] <= 8 else None
        else:
            state["v"] = _normal(gen, *k.shape).to(kind)
            if case["ragged"]:
                state["v"][past] = float("nan")
            state["go"] = _normal(gen, *q.shape).to(kind)
            state["lists"] = _lists(state, _summaries(state["k"], state["length"], BLOCK))
    return state


# ---- plain forms --------------------------------------------------------------
def _rope_plain(s):
    half = s["dim"] // 2
    axis = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(s["pairs"], device="cuda"))
    axis = torch.nn.functional.pad(axis, (0, half - axis.numel()))
    angle = s["pos"].float()[..., axis] * s["freq"]
    angle = -angle if s["inverse"] else angle
    cos, sin = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]

    def turn(x):
        y = x.float()
        a, b = (y[..., 0::2], y[..., 1::2]) if s["interleaved"] else (y[..., :half], y[..., half:])
        a, b = a * cos - b * sin, a * sin + b * cos
        y = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
        return y.to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _norm_plain(s):
    x, f, kind = s["x"].float(), s["f"].float(), s["x"].dtype
    rows, a, eps = s["rows"], s["scale"], s["eps"]
    segment = torch.arange(rows, device="cuda") // s["per_gate"]
    gate = s["gate"][segment]
    r2 = torch.rsqrt((f * f).mean(-1, keepdim=True) + eps)
    fh = f * r2
    y = x + a * gate * (fh * s["w_post"])
    r1 = torch.rsqrt((y * y).mean(-1, keepdim=True) + eps)
    yh = y * r1
    out = [y.to(kind), (yh * s["w_pre"]).to(kind)]
    if s["train"]:
        gy, gh = s["gy"].float(), s["gh"].float()
        d1 = gh * s["w_pre"]
        t = gy + r1 * (d1 - yh * (d1 * yh).mean(-1, keepdim=True))
        d2 = a * t * gate * s["w_post"]
        gf = r2 * (d2 - fh * (d2 * fh).mean(-1, keepdim=True))
        along = a * t * fh
        short = s["gate"].shape[0] * s["per_gate"] - rows
        by_gate = torch.nn.functional.pad(along, (0, 0, 0, short)).unflatten(0, (-1, s["per_gate"])).sum(1)
        out += [t.to(kind), gf.to(kind), by_gate * s["w_post"], (by_gate * s["gate"]).sum(0), (gh * yh).sum(0)]
    return out


def _valid(lk, length, batch):
    """[batch][lk]: the keys that are there."""
    at = torch.arange(lk, device="cuda")[None].expand(batch, lk)
    return at < (lk if length is None else length[:, None])


def _summaries(x, length, size):
    """8-bit means of blocks of `size` tokens, [b][h][blocks][d], and their scales."""
    b, n, h, d = x.shape
    there = _valid(n, length, b)
    fixed = torch.nan_to_num(x.float() * 256.0, nan=0.0).round().clamp(-32768.0, 32768.0)
    fixed = torch.where(there[:, :, None, None], fixed, 0.0)
    pad = -n % size
    total = torch.nn.functional.pad(fixed, (0, 0, 0, 0, 0, pad)).unflatten(1, (-1, size)).sum(2).int().transpose(1, 2)
    count = torch.nn.functional.pad(there, (0, pad)).unflatten(1, (-1, size)).sum(2)
    largest = total.abs().amax(-1, keepdim=True)
    shift = (torch.frexp(largest.float())[1] - 7).clamp_min(0)
    eight = ((total + ((1 << shift) >> 1)) >> shift).clamp_max(127).to(torch.int8)
    scale = torch.ldexp(1.0 / count.clamp_min(1).float()[:, None], shift[..., 0])
    return eight, scale


def _lists(s, summary):
    """The ids of the chosen key blocks, ascending, -1 after the last."""
    b, lq, lk, hq, hk, top = (s[n] for n in ("batch", "lq", "lk", "hq", "hk", "top"))
    length = torch.full((b,), lk, device="cuda") if s["length"] is None else s["length"].long()
    eight, scale = (x.repeat_interleave(hq // hk, 1) for x in summary)
    query = _summaries(s["q"], None, GROUP)[0]
    groups, blocks = query.shape[2], eight.shape[2]
    score = (query.float() @ eight.float().transpose(-1, -2).contiguous()) * scale[:, :, None]
    block = torch.arange(blocks, device="cuda")
    first = torch.arange(groups, device="cuda") * GROUP
    last = (first + GROUP).clamp_max(lq) - 1
    seen = length[:, None].expand(b, groups)
    if s["causal"]:
        low, high = first + (length - lq)[:, None], last + (length - lq)[:, None]
        seen = torch.minimum(seen, high + 1)
        held = (block >= low[..., None].clamp_min(0) // BLOCK) & (block * BLOCK <= high[..., None])
        score = torch.where(held[:, None], float("inf"), score)
    score = torch.where((block * BLOCK < seen[..., None])[:, None], score, float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True)
    ids = torch.where(order.values > float("-inf"), order.indices, blocks)[..., :top].sort(-1).values
    ids = torch.nn.functional.pad(ids, (0, top - ids.shape[-1]), value=blocks)
    return torch.where(ids < blocks, ids, -1).int()


def _attend_plain(s):
    b, lq, lk, hq, hk, dim = (s[n] for n in ("batch", "lq", "lk", "hq", "hk", "dim"))
    kind, soft, lists = s["q"].dtype, dim ** -0.5, s["lists"].long()
    groups, top = lists.shape[2], lists.shape[3]
    blocks = (lk + BLOCK - 1) // BLOCK
    there = _valid(lk, s["length"], b)

    def by_group(x):
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, groups * GROUP - lq))
        return x.unflatten(1, (groups, GROUP)).permute(0, 3, 1, 2, 4)

    def by_block(x):
        x = torch.where(there[:, :, None, None], x.float(), 0.0)
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, blocks * BLOCK - lk))
        return x.unflatten(1, (blocks, BLOCK)).permute(0, 3, 1, 2, 4).reshape(b * hk * blocks, BLOCK, dim)

    head = torch.arange(b * hq, device="cuda").view(b, hq, 1, 1)
    head = head // hq * hk + head % hq // (hq // hk)
    at = (head * blocks + lists.clamp_min(0)).flatten()

    def gathered(x):
        return x[at].view(b, hq, groups, top * BLOCK, dim)

    key = lists.clamp_min(0)[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")
    length = torch.full((b,), lk, device="cuda") if s["length"] is None else s["length"].long()
    sees = ((key < length.view(b, 1, 1, 1, 1)) & (lists[..., None] >= 0)).flatten(-2)[..., None, :]
    if s["causal"]:
        query = torch.arange(groups * GROUP, device="cuda").view(1, 1, groups, GROUP, 1)
        sees = sees & (key.flatten(-2)[..., None, :] <= query + (length - lq).view(b, 1, 1, 1, 1))
    q, k, v = by_group(s["q"]), gathered(by_block(s["k"])), gathered(by_block(s["v"]))
    score = torch.where(sees, (q @ k.transpose(-1, -2)) * soft, float("-inf"))
    top_score = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top_score > float("-inf"), top_score, 0.0))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    out = p @ v

    def tokens(x):
        return x.permute(0, 2, 3, 1, 4).reshape(b, groups * GROUP, hq, dim)[:, :lq].to(kind)

    lse = (top_score + torch.log(total))[..., 0].flatten(2)[..., :lq]
    results = [tokens(out), lse]
    if s["train"]:
        go = by_group(s["go"])
        d = p * (go @ v.transpose(-1, -2) - (go * out).sum(-1, keepdim=True))

        def to_blocks(x):
            x = x.reshape(-1, BLOCK * dim)
            x = torch.zeros(b * hk * blocks, BLOCK * dim, device="cuda").index_add_(0, at, x)
            return x.view(b, hk, blocks * BLOCK, dim)[:, :, :lk].transpose(1, 2).to(kind).contiguous()

        results += [tokens(d @ k * soft), to_blocks(d.transpose(-1, -2) @ q * soft), to_blocks(p.transpose(-1, -2) @ go)]
    return results


def _plain(s):
    if s["op"] == "rope":
        return _rope_plain(s)
    if s["op"] == "norm":
        return _norm_plain(s)
    if s["op"] == "attend":
        return _attend_plain(s)
    summary = s["summary"] or _summaries(s["k"], s["length"], BLOCK)
    return (_lists(s, summary),) + (() if s["summary"] else (summary[0] * summary[1][..., None],))


# ---- the framework's calls ----------------------------------------------------
def _framework(s):
    from gaussian_splatting_differentiable_ewa_amd import tokens as T

    if s["op"] == "rope":
        return T.rope_axes(s["q"], s["k"], s["pos"], s["freq"], s["pairs"], interleaved=s["interleaved"],
                           inverse=s["inverse"])
    if s["op"] == "norm":
        y, h, stats = T.norm_gate(s["x"], s["f"], s["gate"], s["w_post"], s["w_pre"], scale=s["scale"], eps=s["eps"],
                                  rows_per_gate=s["per_gate"])
        if not s["train"]:
            return [y, h]
        return [y, h, *T.norm_gate_backward(s["gy"], s["gh"], s["x"], s["f"], s["gate"], s["w_post"], s["w_pre"], stats,
                                            scale=s["scale"], rows_per_gate=s["per_gate"])]
    if s["op"] == "select":
        summary = s["summary"] or T.block_summary(s["k"], kv_len=s["length"])
        lists = T.select_blocks(s["q"], summary, s["lk"], s["top"], kv_len=s["length"], causal=s["causal"])
        return (lists,) + (() if s["summary"] else (summary[0] * summary[1][..., None],))
    out, lse = T.block_attention(s["q"], s["k"], s["v"], s["lists"], kv_len=s["length"], causal=s["causal"])
    if not s["train"]:
        return [out, lse]
    return [out, lse, *T.block_attention_backward(s["go"], s["q"], s["k"], s["v"], out, lse, s["lists"],
                                                  kv_len=s["length"], causal=s["causal"])]


def run(state):
    return _framework(state) if own else _plain(state)


# ---- what a pass cannot do without --------------------------------------------
def work(case):
    size = BYTES[case["type"]]
    if case["op"] == "rope":
        values = case["batch"] * case["tokens"] * (case["hq"] + case["hk"]) * case["dim"]
        return {"bytes": 2 * size * values + 12 * case["batch"] * case["tokens"], "flops": 3 * values}
    if case["op"] == "norm":
        values = case["rows"] * case["channels"]
        # forward: x, f in, y, h out; backward: x, f, gy, gh in, gx, gf out (x and f read once for both)
        return {"bytes": size * values * (8 if case["train"] else 4), "flops": values * (35 if case["train"] else 10)}
    b, lq, lk, hq, hk, dim, top = (case[n] for n in ("batch", "lq", "lk", "hq", "hk", "dim", "top"))
    groups, blocks = (lq + GROUP - 1) // GROUP, (lk + BLOCK - 1) // BLOCK
    queries, keys = size * b * lq * hq * dim, size * b * lk * hk * dim
    if case["op"] == "select":
        summary = b * hk * blocks * (dim + 4)
        read = queries + (summary if lq <= 8 else keys + 5 * summary) + 4 * b * hq * groups * top
        return {"bytes": read, "flops": 2 * b * hq * groups * blocks * dim}
    taken = min(top, blocks)
    pairs = b * hq * lq * BLOCK * taken
    if case["causal"] and lq > 1:  # what a causal list can hold, on average over the queries
        seen = min(1.0, sum(min(taken, (lk - lq + g * GROUP) // BLOCK + 2) for g in range(groups)) / (groups * taken))
        pairs = int(pairs * seen)
    touched = size * BLOCK * dim * min(b * hk * blocks, b * hq * groups * taken)
    total = 2 * queries + 2 * touched + 4 * b * hq * (lq + groups * top)
    if not case["train"]:
        return {"bytes": total, "flops": 4 * dim * pairs}
    return {"bytes": total + 2 * queries + 2 * keys, "flops": 14 * dim * pairs}


# ---- the definitions in 64 bits -----------------------------------------------
def _exact_rope(s):
    out = []
    for x in (s["q"].double(), s["k"].double()):
        y = x.clone()
        j = 0
        for axis, count in enumerate(s["pairs"]):
            for _ in range(count):
                t = s["pos"][..., axis].double() * s["freq"][j].double() * (-1 if s["inverse"] else 1)
                c, n = t.cos()[..., None], t.sin()[..., None]
                i0, i1 = (2 * j, 2 * j + 1) if s["interleaved"] else (j, j + s["dim"] // 2)
                y[..., i0] = c * x[..., i0] - n * x[..., i1]
                y[..., i1] = n * x[..., i0] + c * x[..., i1]
                j += 1
        out.append(y)
    return tuple(out)


def _exact_norm(s):
    # the gradients by differentiating the forward formula
    leaves = [s[n].double().requires_grad_() for n in ("x", "f", "gate", "w_post", "w_pre")]
    x, f, gate, w_post, w_pre = leaves
    wide = gate.repeat_interleave(s["per_gate"], 0)[: s["rows"]]
    y = x + s["scale"] * wide * w_post * f / (f.pow(2).mean(1, keepdim=True) + s["eps"]).sqrt()
    h = w_pre * y / (y.pow(2).mean(1, keepdim=True) + s["eps"]).sqrt()
    if not s["train"]:
        return [y.detach(), h.detach()]
    return [y.detach(), h.detach(), *torch.autograd.grad([y, h], leaves, [s["gy"].double(), s["gh"].double()])]


def _exact_summary(x, length, size):
    """Block by block, in whole numbers."""
    b, n, h, d = x.shape
    fixed = (torch.nan_to_num(x.double()) * 256).round().clamp(-32768, 32768).long()
    eight, scale = [], []
    for i in range(0, n, size):
        j = min(n, i + size)
        upto = torch.full((b,), j, device="cuda") if length is None else length.long().clamp(i, j)
        mine = torch.arange(i, j, device="cuda")[None] < upto[:, None]
        total = (fixed[:, i:j] * mine[:, :, None, None]).sum(1)
        shift = torch.zeros(b, h, 1, dtype=torch.long, device="cuda")
        for bit in range(7, 40):
            shift += (total.abs().amax(-1, keepdim=True) >= 1 << bit).long()
        half = torch.where(shift > 0, 1 << (shift - 1).clamp_min(0), 0)
        eight.append(((total + half) >> shift).clamp_max(127))
        inverse = (1.0 / (upto - i).clamp_min(1).double()).float().double()
        scale.append(inverse[:, None] * (1 << shift[..., 0]).double())
    return torch.stack(eight, 2), torch.stack(scale, 2)


def _exact_select(s):
    b, lq, lk, hq, hk, top = (s[n] for n in ("batch", "lq", "lk", "hq", "hk", "top"))
    eight, scale = _exact_summary(s["k"], s["length"], BLOCK)
    query = _exact_summary(s["q"], None, GROUP)[0]
    groups, blocks = query.shape[2], eight.shape[2]
    if b * hq * groups > 5000:
        return None
    lists = torch.full((b, hq, groups, top), -1, dtype=torch.int32)
    for i in range(b):
        n = lk if s["length"] is None else int(s["length"][i])
        for h in range(hq):
            # the score is the 32-bit product of the dot product and the scale
            dots = query[i, h].double() @ eight[i, h * hk // hq].double().T.contiguous()
            scores = (dots.float() * scale[i, h * hk // hq].float()).cpu().tolist()
            for g in range(groups):
                low = g * GROUP + n - lq
                high = min(lq, g * GROUP + GROUP) - 1 + n - lq
                upto = min(n, high + 1) if s["causal"] else n
                seen = range(max(0, (upto + BLOCK - 1) // BLOCK))
                held = [s["causal"] and e * BLOCK <= high and e * BLOCK + BLOCK > low for e in range(blocks)]
                best = sorted(seen, key=lambda e: (not held[e], 0.0 if held[e] else -scores[g][e], e))[:top]
                if best:
                    lists[i, h, g, : len(best)] = torch.tensor(sorted(best), dtype=torch.int32)
    lists = lists.cuda()
    return (lists,) if s["summary"] else (lists, eight.double() * scale[..., None])


def _exact_attend(s):
    # one head at a time, dense, in bands of queries
    b, lq, lk, hq, hk, dim = (s[n] for n in ("batch", "lq", "lk", "hq", "hk", "dim"))
    if b * hq * lq * lk > 16 * 33000 ** 2:
        return None
    blocks = (lk + BLOCK - 1) // BLOCK
    band = max(GROUP, (1 << 28) // lk // GROUP * GROUP)
    out = torch.zeros(b, lq, hq, dim, dtype=torch.double, device="cuda")
    lse = torch.zeros(b, hq, lq, dtype=torch.double, device="cuda")
    gq, gk, gv = (torch.zeros(b, n, h, dim, dtype=torch.double, device="cuda") for n, h in ((lq, hq), (lk, hk), (lk, hk)))
    for i in range(b):
        n = lk if s["length"] is None else int(s["length"][i])
        for h in range(hq):
            k, v = s["k"][i, :n, h * hk // hq].double(), s["v"][i, :n, h * hk // hq].double()
            for lo in range(0, lq, band):
                hi = min(lq, lo + band)
                q = s["q"][i, lo:hi, h].double()
                ids = s["lists"][i, h, lo // GROUP: (hi + GROUP - 1) // GROUP].long()
                on = torch.zeros(ids.shape[0], blocks + 1, dtype=torch.bool, device="cuda")
                on.scatter_(1, torch.where(ids >= 0, ids, blocks), True)
                mask = on[:, :blocks].repeat_interleave(GROUP, 0)[: hi - lo].repeat_interleave(BLOCK, 1)[:, :n]
                if s["causal"]:
                    limit = torch.arange(lo, hi, device="cuda")[:, None] + n - lq
                    mask = mask & (torch.arange(n, device="cuda")[None] <= limit)
                w = (q @ k.T.contiguous() / math.sqrt(dim)).masked_fill(~mask, float("-inf"))
                z = torch.logsumexp(w, 1)
                lse[i, h, lo:hi] = z
                w = torch.exp(w - z.masked_fill(z == float("-inf"), 0.0)[:, None])
                o = w @ v
                out[i, lo:hi, h] = o
                if s["train"]:
                    g = s["go"][i, lo:hi, h].double()
                    gv[i, :n, h * hk // hq] += w.T.contiguous() @ g
                    w = w * (g @ v.T.contiguous() - (g * o).sum(1, keepdim=True)) / math.sqrt(dim)
                    gq[i, lo:hi, h] = w @ k
                    gk[i, :n, h * hk // hq] += w.T.contiguous() @ q
    return [out, lse, gq, gk, gv] if s["train"] else [out, lse]


def exact(case, seed):
    state = prepare(case, seed)
    return {"rope": _exact_rope, "norm": _exact_norm, "select": _exact_select, "attend": _exact_attend}[case["op"]](state)
