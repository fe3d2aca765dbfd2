"""A small network that predicts Gaussians from posed views, built from the token
operators and trained through the rasterizer.

Every 16x16 tile of every view is a token. A layer is attention over the key
blocks that ``select_blocks`` chooses (queries and keys turned by their (view,
row, column) positions) and a two-layer perceptron; after each, ``NormGate``
norms the result, gates and scales it into the residual stream and norms that
for the next. The head places ``per_tile`` Gaussians per token along the tile's
camera rays (SH degree 0, 14 parameters); ``RenderL1`` renders them with
``gs_preprocess``, ``gs_tile_lists`` and ``gs_rasterize_fwd_bwd_l1`` and hands
the parameters' gradients back. Linear layers are plain library products.

``TileNet.forward`` takes all views at once (training), each attending to every
view or, with ``causal``, to itself and the views before it; ``TileNet.extend``
takes the next view against a ``TileCache`` of the views seen so far (serving)
and computes what the causal form does: its keys, values and block summaries
are kept, and only the blocks it touches are summarised again. ``train`` fits
the causal form unless told otherwise.

``gated`` makes the perceptron a gated one (``GatedFF``), ``layer_norm`` norms a
tile's pixels before the embedding (``LayerNorm``), and ``pack4`` holds the
layers' weights in 4 bits for ``extend`` (``linear4``), at a quarter of the bytes.

    python -m gaussian_splatting_differentiable_ewa_amd.predictor --steps 60
"""

from __future__ import annotations

import argparse
import math
from typing import List, Optional, Sequence, Tuple

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

from . import _lib as L
from . import tokens as T
from .step import Buffers

PARAMS = 14  # Gaussian parameters at SH degree 0
DIM = 64     # of a head


class RenderL1(torch.autograd.Function):
    """apply(params, buf, target) -> mean absolute error of the rendered views
    (``buf``: step.Buffers of the cameras; target [V][3][H][W])."""

    @staticmethod
    def forward(ctx, params, buf, target):
        params = params.contiguous()
        buf.preprocess(params)
        buf.intersections()
        buf.rasterize_fwd_bwd_l1(target, image=True, accumulate_grad2d=True)
        grad = torch.empty_like(params)
        L.gs_preprocess_bwd(params, buf.n, buf.sh_degree, buf.cams, buf.rect, buf.grad2d, grad)
        ctx.save_for_backward(grad)
        return buf.loss[0].float()

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        return ctx.saved_tensors[0] * g, None, None


class TileCache:
    """Keys, values and block summaries of the views seen so far, for every
    layer, with room for ``capacity`` tokens."""

    def __init__(self, layers: int, capacity: int, heads: int, dtype=torch.bfloat16, device="cuda"):
        self.capacity, self.tokens, self.views = capacity, 0, 0
        self.length = torch.zeros(1, dtype=torch.int32, device=device)
        blocks = (capacity + T.BLOCK - 1) // T.BLOCK
        self.k = [torch.empty(1, capacity, heads, DIM, dtype=dtype, device=device) for _ in range(layers)]
        self.v = [torch.empty(1, capacity, heads, DIM, dtype=dtype, device=device) for _ in range(layers)]
        # block by block, as the cache grows
        self.sums = [(torch.zeros(1, blocks, heads, DIM, dtype=torch.int8, device=device).transpose(1, 2),
                      torch.zeros(1, blocks, heads, dtype=torch.float32, device=device).transpose(1, 2))
                     for _ in range(layers)]


class TileNet(torch.nn.Module):
    """Views [V, 3, H, W] -> Gaussian parameters [14][V x tiles x per_tile]."""

    def __init__(self, channels: int = 256, heads: int = 4, kv_heads: int = 2, layers: int = 2, per_tile: int = 4,
                 top: int = 16, views: int = L.GS_MAX_VIEWS, depth: float = 8.0, dtype=torch.bfloat16, seed: int = 0,
                 hidden: Optional[int] = None, gated: Optional[str] = None, layer_norm: bool = False):
        super().__init__()
        hidden = 4 * channels if hidden is None else hidden
        if channels % 8 or hidden % 8 or heads % kv_heads:
            raise ValueError("channels and hidden must be multiples of 8 and heads of kv_heads")
        if gated is not None and gated not in T.ACTS:
            raise ValueError(f"gated must be None or one of {sorted(T.ACTS)}, got {gated!r}")
        self.channels, self.heads, self.kv_heads, self.layers = channels, heads, kv_heads, layers
        self.per_tile, self.top, self.depth, self.dtype, self.views = per_tile, top, depth, dtype, views
        self.gated = gated
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, scale=1.0):
            return torch.nn.Parameter(torch.randn(*shape, generator=g) * (scale / math.sqrt(shape[-1])))

        c, tile = channels, 3 * L.GS_TILE ** 2
        self.embed = weight(c, tile)
        self.first = torch.nn.Parameter(torch.ones(c))
        self.qkv = torch.nn.ParameterList([weight((heads + 2 * kv_heads) * DIM, c) for _ in range(layers)])
        self.out = torch.nn.ParameterList([weight(c, heads * DIM) for _ in range(layers)])
        self.up = torch.nn.ParameterList([weight(hidden, c) for _ in range(layers)])
        self.down = torch.nn.ParameterList([weight(c, hidden) for _ in range(layers)])
        # norms after and before, and the gate of each view, of 2 blocks a layer
        self.post = torch.nn.ParameterList([torch.nn.Parameter(torch.ones(c)) for _ in range(2 * layers)])
        self.pre = torch.nn.ParameterList([torch.nn.Parameter(torch.ones(c)) for _ in range(2 * layers)])
        self.gate = torch.nn.ParameterList([torch.nn.Parameter(torch.ones(views, c)) for _ in range(2 * layers)])
        self.head = weight(per_tile * PARAMS, c, scale=0.1)
        if gated is not None:  # the projection that opens and closes `up`'s
            self.open = torch.nn.ParameterList([weight(hidden, c) for _ in range(layers)])
        self.pixels = torch.nn.ParameterList([torch.nn.Parameter(f(tile)) for f in (torch.ones, torch.zeros)] if layer_norm else [])
        self.pairs = (8, 12, 12)  # of the 32 pairs of a head: view, row, column
        self.register_buffer("freq", torch.cat([100.0 ** (-torch.arange(p, dtype=torch.float32) / p) for p in self.pairs]))

    # ---- tokens -------------------------------------------------------------
    def _tiles(self, images):
        """[V, 3, H, W] -> [V x TY x TX, 768], zeros past the image's edge."""
        v, _, h, w = images.shape
        t = L.GS_TILE
        x = F.pad(images, (0, -w % t, 0, -h % t)).unflatten(3, (-1, t)).unflatten(2, (-1, t))
        return x.permute(0, 2, 4, 1, 3, 5).reshape(-1, 3 * t * t).to(self.dtype)

    def _positions(self, first_view, views, ty, tx, device):
        at = torch.arange(views * ty * tx, device=device)
        return torch.stack([at // (ty * tx) + first_view, at // tx % ty, at % tx], -1).int()[None]

    def _linear(self, x, w, four=None):
        return x @ w.to(self.dtype).t() if four is None else T.linear4(x, four)

    def _perceptron(self, i, h, four):
        if self.gated is None:
            return self._linear(F.gelu(self._linear(h, self.up[i], four.get("up"))), self.down[i], four.get("down"))
        if not four:
            weights = (w[i].to(self.dtype) for w in (self.open, self.up, self.down))
            return (T.GatedFF.apply if torch.is_grad_enabled() else T.gated_ff)(h, *weights, self.gated)
        opened, up = T.linear4(h, four["open up"]).chunk(2, 1)
        return T.linear4(getattr(F, self.gated)(opened) * up, four["down"])

    def pack4(self) -> List[dict]:
        """The layers' weights in 4 bits, for ``extend`` (channels, hidden and the
        heads' width have to be multiples of 32); the embedding and the head stay
        in 16."""
        layers = []
        for i in range(self.layers):
            of = {"qkv": self.qkv[i], "out": self.out[i], "down": self.down[i]}
            if self.gated is None:
                of["up"] = self.up[i]
            else:
                of["open up"] = torch.cat([self.open[i], self.up[i]])
            layers.append({name: T.quantise4(w.detach().to(self.dtype)) for name, w in of.items()})
        return layers

    def _layers(self, tiles, pos, per_view, first_view, attend, four=None):
        """Residual stream's norm after all layers; attend(layer, q, k, v)."""
        n, views = tiles.shape[0], tiles.shape[0] // per_view
        four = [{}] * self.layers if four is None else four
        if len(self.pixels):
            tiles = T.LayerNorm.apply(tiles, *self.pixels)
        x, h = T.NormGate.apply(self._linear(tiles, self.embed), None, None, None, self.first)
        scale = 1.0 / math.sqrt(2 * self.layers)
        for i in range(self.layers):
            q, k, v = self._linear(h, self.qkv[i], four[i].get("qkv")).view(1, n, -1, DIM).split([self.heads, self.kv_heads, self.kv_heads], 2)
            q, k = T.RopeAxes.apply(q, k, pos, self.freq, self.pairs)
            f = self._linear(attend(i, q, k, v).reshape(n, -1), self.out[i], four[i].get("out"))
            gates = self.gate[2 * i][first_view: first_view + views].contiguous()
            x, h = T.NormGate.apply(x, f, gates, self.post[2 * i], self.pre[2 * i], scale, 1e-6, per_view)
            f = self._perceptron(i, h, four[i])
            gates = self.gate[2 * i + 1][first_view: first_view + views].contiguous()
            x, h = T.NormGate.apply(x, f, gates, self.post[2 * i + 1], self.pre[2 * i + 1], scale, 1e-6, per_view)
        return h

    # ---- Gaussians ------------------------------------------------------------
    def _gaussians(self, h, cams, ty, tx):
        """Tokens to parameters: per Gaussian an offset in its tile, a depth on
        that ray, scales relative to the tile's size there, and the rest."""
        v, g, t = len(cams), self.per_tile, L.GS_TILE
        raw = (h @ self.head.to(self.dtype).t()).float().view(v, ty * tx, g, PARAMS)
        dev = raw.device
        cam = torch.tensor([[c.fx, c.fy, c.cx, c.cy] for c in cams], device=dev)
        R = torch.tensor([c.R for c in cams], device=dev).view(v, 3, 3)
        shift = torch.tensor([c.t for c in cams], device=dev)
        fx, fy, cx, cy = (cam[:, i].view(v, 1, 1) for i in range(4))
        side = int(math.ceil(math.sqrt(g)))  # the Gaussians of a tile start on a grid
        spot = torch.arange(g, device=dev)
        at = torch.arange(ty * tx, device=dev).view(1, -1, 1)
        u = (at % tx) * t + t * (spot % side + 0.5) / side + t * torch.tanh(raw[..., 0])
        w = (at // tx) * t + t * (spot // side + 0.5) / side + t * torch.tanh(raw[..., 1])
        z = self.depth * torch.exp(raw[..., 2])
        p = torch.stack([(u - cx) / fx * z, (w - cy) / fy * z, z], -1) - shift.view(v, 1, 1, 3)
        mean = (p.flatten(1, 2).unsqueeze(-1) * R.unsqueeze(1)).sum(2).view(v, -1, g, 3)  # R^T p
        size = torch.log(z * t / (2 * side * fx))
        scales = size.unsqueeze(-1) + raw[..., 3:6]
        quat = raw[..., 6:10] + torch.tensor([1.0, 0, 0, 0], device=dev)
        return torch.cat([mean, scales, quat, raw[..., 10:11] + 1.0, raw[..., 11:14]], -1).flatten(0, 2).t()

    def forward(self, images, cams: Sequence, causal: bool = False):
        """causal: a view attends to itself and the views before it, as in
        ``extend``; else every view to all of them."""
        v, _, h, w = images.shape
        ty, tx = (h + L.GS_TILE - 1) // L.GS_TILE, (w + L.GS_TILE - 1) // L.GS_TILE
        n = ty * tx
        pos = self._positions(0, v, ty, tx, images.device)

        def attend(i, q, k, v):
            with torch.no_grad():
                lists = T.select_blocks(q, T.block_summary(k), k.shape[1], self.top)
            return T.BlockAttention.apply(q, k, v, lists)

        def attend_by_view(i, q, k, v):
            # its groups of queries begin with the view, and the summaries hold no later view's keys
            blocks = (k.shape[1] + T.BLOCK - 1) // T.BLOCK
            eight = torch.empty(1, self.kv_heads, blocks, DIM, dtype=torch.int8, device=k.device)
            scale = torch.empty(1, self.kv_heads, blocks, dtype=torch.float32, device=k.device)
            out = []
            for before in range(0, k.shape[1], n):
                upto = before + n
                blocks = (upto + T.BLOCK - 1) // T.BLOCK
                mine, sums = q[:, before:upto], (eight[:, :, :blocks], scale[:, :, :blocks])
                with torch.no_grad():
                    T.block_summary(k[:, :upto], None, sums, before // T.BLOCK)
                    lists = T.select_blocks(mine, sums, upto, self.top)
                out.append(T.BlockAttention.apply(mine, k[:, :upto], v[:, :upto], lists))
            return torch.cat(out, 1)

        h = self._layers(self._tiles(images), pos, n, 0, attend_by_view if causal else attend)
        return self._gaussians(h, cams, ty, tx)

    @torch.no_grad()
    def extend(self, image, cam, cache: TileCache, four: Optional[List[dict]] = None):
        """The Gaussians of the next view ([3, H, W]), its tokens attending to
        themselves and to all views before it. Views may differ in size: the cache
        counts them. four: ``pack4``'s weights instead of the network's own."""
        _, h, w = image.shape
        ty, tx = (h + L.GS_TILE - 1) // L.GS_TILE, (w + L.GS_TILE - 1) // L.GS_TILE
        n, before, view = ty * tx, cache.tokens, cache.views
        if before + n > cache.capacity:
            raise ValueError(f"the cache holds {cache.capacity} tokens, {before + n} are needed")
        if view >= self.views:
            raise ValueError(f"the network has gates for {self.views} views, and the cache holds {view}")
        pos = self._positions(view, 1, ty, tx, image.device)
        cache.length.fill_(before + n)
        first = before // T.BLOCK
        blocks = (before + n + T.BLOCK - 1) // T.BLOCK - first

        def attend(i, q, k, v):
            cache.k[i][:, before: before + n] = k
            cache.v[i][:, before: before + n] = v
            T.block_summary(cache.k[i], cache.length, cache.sums[i], first, blocks)
            # the length hides what comes after the view; inside it every tile sees every other
            lists = T.select_blocks(q, cache.sums[i], cache.capacity, self.top, cache.length)
            return T.block_attention(q, cache.k[i], cache.v[i], lists, None, cache.length)[0]

        tokens = self._layers(self._tiles(image[None]), pos, n, view, attend, four)
        cache.tokens, cache.views = before + n, view + 1
        return self._gaussians(tokens, [cam], ty, tx)


def train(images, cams: Sequence, steps: int = 60, lr: float = 2e-3, net: Optional[TileNet] = None,
          report=None, causal: bool = True) -> Tuple[TileNet, List[float]]:
    """Fits a network to posed views; the network and the loss of every step.
    causal: in the form that ``extend`` serves; else with every view seeing all."""
    net = (net or TileNet()).to(images.device)
    v, _, h, w = images.shape
    tiles = ((h + L.GS_TILE - 1) // L.GS_TILE) * ((w + L.GS_TILE - 1) // L.GS_TILE)
    buf = Buffers(v * tiles * net.per_tile, 0, cams, device=images.device)
    adam = torch.optim.Adam(net.parameters(), lr=lr)
    losses = []
    for s in range(steps):
        loss = RenderL1.apply(net(images, cams, causal=causal), buf, images)
        adam.zero_grad(set_to_none=True)
        loss.backward()
        adam.step()
        losses.append(float(loss.detach()))
        if report is not None and (s % 10 == 0 or s == steps - 1):
            report(f"step {s}: L1 {losses[-1]:.5f}")
    return net, losses


def main(argv=None):
    from . import scenes
    from .step import render

    p = argparse.ArgumentParser(description="Fit a tile network to rendered views of a synthetic scene.")
    p.add_argument("--config", type=int, default=0, help="scene of scenes.CONFIGS (0: 256x256, 10k Gaussians)")
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--gated", choices=sorted(T.ACTS), help="a gated perceptron with this activation")
    p.add_argument("--layer-norm", action="store_true", help="norm the tiles' pixels before the embedding")
    a = p.parse_args(argv)
    cfg = scenes.CONFIGS[a.config]
    cams = cfg.cameras()
    params = torch.from_numpy(scenes.make_params(cfg)).cuda()
    images = render(params, cfg.sh_degree, cams).clone()
    train(images, cams, a.steps, net=TileNet(gated=a.gated, layer_norm=a.layer_norm), report=print)


if __name__ == "__main__":
    main()
