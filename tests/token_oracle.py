"""The token operators from their definitions in 64 bits, one sequence and head
at a time, for the GPU tests. Each also returns what its error bound is made
of: the sums of magnitudes that roundings are relative to."""

import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half an ulp, relative
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the least subnormal
E = 2.0 ** -24


def rope(x, pos, freq, pairs, interleaved, inverse):
    """(turned x, |x0| + |x1| of each element's pair)."""
    x = x.double()
    out, mag = x.clone(), x.abs()
    half = x.shape[-1] // 2
    j = 0
    for axis, n in enumerate(pairs):
        for _ in range(n):
            t = pos[..., axis].double() * freq[j].double()
            c, s = torch.cos(t)[..., None], torch.sin(t)[..., None] * (-1 if inverse else 1)
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            out[..., a] = x[..., a] * c - x[..., b] * s
            out[..., b] = x[..., a] * s + x[..., b] * c
            mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
            j += 1
    return out, mag


def norm_gate(x, f, gate, w_post, w_pre, scale, eps, per):
    x = x.double()
    if f is not None:
        f = f.double()
        g = torch.ones_like(x) if gate is None else gate.double().repeat_interleave(per, 0)[: x.shape[0]]
        g = g * (1.0 if w_post is None else w_post.double())
        x = x + scale * g * f / torch.sqrt((f * f).mean(-1, keepdim=True) + eps)
    h = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x, h * (1.0 if w_pre is None else w_pre.double())


def summary(x, size, length=None):
    """(sum8, scale) in whole numbers, [batch][heads][blocks]."""
    b, n, h, d = x.shape
    blocks = (n + size - 1) // size
    fixed = torch.nan_to_num(x.double() * 256, nan=0.0).round().clamp(-32768, 32768).long()
    eight = torch.zeros(b, h, blocks, d, dtype=torch.long, device=x.device)
    scale = torch.zeros(b, h, blocks, dtype=torch.double, device=x.device)
    for i in range(b):
        end = n if length is None else max(0, min(n, int(length[i])))
        for m in range(blocks):
            lo, hi = m * size, max(m * size, min(end, (m + 1) * size))
            total = fixed[i, lo:hi].sum(0)
            e = (total.abs().amax(-1) if d else total.sum(-1)).tolist()
            for k in range(h):
                shift = max(0, int(e[k]).bit_length() - 7)
                eight[i, k, m] = ((total[k] + ((1 << shift) >> 1)) >> shift).clamp_max(127)
                scale[i, k, m] = float(torch.tensor(1.0 / max(1, hi - lo), dtype=torch.float32)) * 2.0 ** shift
    return eight, scale


def select(q, sums, tokens_k, top, length=None, causal=False):
    b, n, h, d = q.shape
    eight, scale = sums
    q8 = summary(q, 128)[0]
    groups = q8.shape[2]
    out = torch.full((b, h, groups, top), -1, dtype=torch.int32)
    for i in range(b):
        end = tokens_k if length is None else max(0, min(tokens_k, int(length[i])))
        for k in range(h):
            kk = k * eight.shape[1] // h
            dots = q8[i, k].double() @ eight[i, kk].double().T.contiguous()
            scores = (dots.float() * scale[i, kk].float()).tolist()
            for g in range(groups):
                low, high = g * 128 + end - n, min(n, g * 128 + 128) - 1 + end - n
                seen = min(end, high + 1) if causal else end
                ids = range((seen + 63) // 64 if seen > 0 else 0)
                own = [causal and m * 64 <= high and m * 64 + 64 > low for m in range(eight.shape[2])]
                best = sorted(ids, key=lambda m: (not own[m], 0.0 if own[m] else -scores[g][m], m))[:top]
                out[i, k, g, : len(best)] = torch.tensor(sorted(best), dtype=torch.int32)
    return out


def listed(lists, blocks):
    """[groups][blocks] truth values: the entries that count (those that exceed
    the entry before them and lie inside the blocks)."""
    on = torch.zeros(lists.shape[0], blocks, dtype=torch.bool, device=lists.device)
    for g, row in enumerate(lists.tolist()):
        for j, m in enumerate(row):
            if 0 <= m < blocks and m > (row[j - 1] if j else -1):
                on[g, m] = True
    return on


def attention(q, k, v, lists, scale, length=None, causal=False, gout=None):
    """Results and error bounds by name. The bounds follow the stated roundings:
    scores in fp32 (dim products each), probabilities and their gradients
    rounded once to the inputs' type, outputs rounded once."""
    b, n, h, d = q.shape
    tokens, hk = k.shape[1], k.shape[2]
    blocks = (tokens + 63) // 64
    u, tiny, dev = U[q.dtype], TINY[q.dtype], q.device
    z = lambda *s: torch.zeros(*s, dtype=torch.double, device=dev)  # noqa: E731
    r = {"out": z(b, n, h, d), "lse": z(b, h, n), "gq": z(b, n, h, d), "gk": z(b, tokens, hk, d), "gv": z(b, tokens, hk, d)}
    e = {name: torch.zeros_like(x) for name, x in r.items()}
    for i in range(b):
        end = tokens if length is None else max(0, min(tokens, int(length[i])))
        for j in range(h):
            c = j * hk // h
            on = listed(lists[i, j], blocks).repeat_interleave(128, 0)[:n].repeat_interleave(64, 1)[:, :end]
            if causal:
                on = on & (torch.arange(end, device=dev) <= torch.arange(n, device=dev)[:, None] + end - n)
            Q, K, V = q[i, :, j].double(), k[i, :end, c].double(), v[i, :end, c].double()
            S = (Q @ K.T.contiguous() * scale).masked_fill(~on, -math.inf)
            empty = ~on.any(1)
            lse = torch.logsumexp(S, 1) if end else torch.full((n,), -math.inf, dtype=torch.double, device=dev)
            P = torch.exp(S - lse.masked_fill(empty, 0.0)[:, None])
            # a score is d fp32 products and sums, its scaling, the subtraction of the maximum and exp2's ulp
            eS = ((Q.abs() @ K.abs().T.contiguous()) * scale * (d + 4) * E + (S.abs() + lse.abs()[:, None]) * 4 * E + 4 * E)
            eS = eS.masked_fill(~on, 0.0)
            worst = eS.amax(1, keepdim=True) if end else eS.sum(1, keepdim=True)
            eP = P * (2 * worst + end ** 0.5 * 4 * E)  # relative: the score's and the sum's errors, in fp32
            out = P @ V
            r["out"][i, :, j], r["lse"][i, j] = out, lse
            e["out"][i, :, j] = (P * u + eP + tiny) @ V.abs() + u * out.abs() + tiny
            e["lse"][i, j] = torch.where(empty, 0.0, worst[:, 0] + end ** 0.5 * 4 * E + lse.abs() * 4 * E)
            if gout is None:
                continue
            G = gout[i, :, j].double()
            dP, D = G @ V.T.contiguous(), (G * out).sum(1, keepdim=True)
            dS = P * (dP - D)
            eD = (G.abs() * e["out"][i, :, j]).sum(1, keepdim=True) + d * E * (G * out).abs().sum(1, keepdim=True)
            eDP = (G.abs() @ V.abs().T.contiguous()) * (d + 4) * E
            edS = eP * (dP - D).abs() + P * (eD + eDP) + u * dS.abs() + tiny * on
            edS = edS * (1 + u)
            r["gq"][i, :, j] = dS @ K * scale
            e["gq"][i, :, j] = (edS @ K.abs() * scale) * (1 + E * end ** 0.5) + u * r["gq"][i, :, j].abs() + tiny
            r["gk"][i, :end, c] += dS.T.contiguous() @ Q * scale
            e["gk"][i, :end, c] += edS.T.contiguous() @ Q.abs() * scale
            r["gv"][i, :end, c] += P.T.contiguous() @ G
            e["gv"][i, :end, c] += (P * u + eP + tiny * on).T.contiguous() @ G.abs()
    for name in ("gk", "gv"):
        e[name] += (u + 64 * E) * (r[name].abs() + e[name]) + tiny
    return r, e
