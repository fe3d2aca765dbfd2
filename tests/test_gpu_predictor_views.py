"""The network fed view by view is the one that sees all views with each view
attending to itself and those before it, also where the selection has to
choose among the blocks."""

import pytest
import torch

from gaussian_splatting_differentiable_ewa_amd import predictor as P
from gaussian_splatting_differentiable_ewa_amd import scenes as S

pytestmark = pytest.mark.gpu


def some_views(count, w, h, seed=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    images = torch.rand(count, 3, h, w, generator=g, device="cuda")
    return images, [S.look_camera(w, h, 100.0, (0.2 * i, 0.0, 0.0)) for i in range(count)]


def contribution(net, got, whole, cams, h, w):
    """How far `got` is from `whole`, relative to what the network adds to the Gaussians' starting values."""
    ty, tx = (h + 15) // 16, (w + 15) // 16
    with torch.no_grad():
        start = net._gaussians(torch.zeros(len(cams) * ty * tx, net.channels, dtype=net.dtype, device="cuda"), cams, ty, tx)
    return start, lambda cols: float((got[:, cols] - whole[:, cols]).norm() / (whole[:, cols] - start[:, cols]).norm())


def test_a_view_attends_to_all_of_itself():
    images, cams = some_views(1, 120, 90)
    net = P.TileNet(layers=2, top=8).cuda()
    with torch.no_grad():
        whole = net(images, cams)
    got = net.extend(images[0], cams[0], P.TileCache(net.layers, 48, net.kv_heads))
    off = contribution(net, got, whole, cams, 90, 120)[1](slice(None))
    assert off <= 4 * net.layers * 2.0 ** -8, off  # bf16 roundings of a layer's products
    # the last tile's pixels reach the first tile's Gaussians
    images[:, :, 80:, 112:] = 1.0
    moved = net.extend(images[0], cams[0], P.TileCache(net.layers, 48, net.kv_heads))
    assert not torch.equal(moved[:, : net.per_tile], got[:, : net.per_tile])


def test_view_by_view_where_blocks_are_chosen(monkeypatch):
    """Three views of 130 tiles, 2 of up to 7 blocks: the same groups, the same
    lists (but for near ties), and the same Gaussians where those agree."""
    images, cams = some_views(3, 208, 160)
    net = P.TileNet(layers=1, top=2).cuda()
    seen = []
    select = P.T.select_blocks
    monkeypatch.setattr(P.T, "select_blocks", lambda *a, **kw: seen.append(select(*a, **kw)) or seen[-1])
    with torch.no_grad():
        whole = net(images, cams, causal=True)
    at_once, seen[:] = list(seen), []
    cache = P.TileCache(net.layers, 3 * 130, net.kv_heads)
    got = torch.cat([net.extend(images[i], cams[i], cache) for i in range(3)], 1)
    assert [x.shape for x in seen] == [x.shape for x in at_once] == [(1, net.heads, 2, 2)] * 3
    assert all((x >= 0).all() for x in seen[1:]) and any(int(x.max() - x.min()) >= 2 for x in seen)
    same = torch.stack([(x == y).all(-1).all(1)[0] for x, y in zip(seen, at_once)])  # [view][group]
    assert same.float().mean() >= 0.8
    off = contribution(net, got, whole, cams, 160, 208)[1]
    width = 130 * net.per_tile
    for i in range(3):
        for m in range(2):
            if same[i, m]:
                cols = slice(i * width + m * 128 * net.per_tile, i * width + min(130, m * 128 + 128) * net.per_tile)
                assert off(cols) <= 4 * net.layers * 2.0 ** -8, (i, m, off(cols))


def test_training_fits_the_form_that_is_served(monkeypatch):
    images, cams = some_views(2, 64, 64)
    how = []
    forward = P.TileNet.forward
    monkeypatch.setattr(P.TileNet, "forward", lambda self, *a, **kw: how.append(kw) or forward(self, *a, **kw))
    P.train(images, cams, steps=1)
    P.train(images, cams, steps=1, causal=False)
    assert how == [dict(causal=True), dict(causal=False)]


def test_gradients_view_by_view():
    """Two views, the first's Gaussians alone: the second's pixels have no part
    in their gradient, the other way round they have."""
    images, cams = some_views(2, 64, 64)
    net = P.TileNet(layers=1, top=4).cuda()
    images.requires_grad_()
    params = net(images, cams, causal=True)
    half = params.shape[1] // 2
    first, = torch.autograd.grad(params[:, :half].sum(), images, retain_graph=True)
    second, = torch.autograd.grad(params[:, half:].sum(), images)
    assert first[0].any() and not first[1].any()
    assert second[0].any() and second[1].any()
