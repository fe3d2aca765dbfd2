"""A cache numbers its views by counting them, whatever their sizes."""

import pytest
import torch

from gaussian_splatting_differentiable_ewa_amd import predictor as P
from gaussian_splatting_differentiable_ewa_amd import scenes as S

pytestmark = pytest.mark.gpu


def test_views_of_different_sizes_are_numbered_in_turn():
    net = P.TileNet(layers=1, top=8, views=3).cuda()
    numbers = []
    positions = net._positions
    net._positions = lambda first, *a: numbers.append(first) or positions(first, *a)
    cache = P.TileCache(net.layers, 400, net.kv_heads)
    for w, h in ((120, 90), (240, 180), (64, 64)):
        image = torch.rand(3, h, w, generator=torch.Generator(device="cuda").manual_seed(w), device="cuda")
        net.extend(image, S.look_camera(w, h, 100.0, (0.0, 0.0, 0.0)), cache)
    assert numbers == [0, 1, 2]
    assert cache.tokens == 48 + 180 + 16
    # a fourth view has no gates of its own: refused before the cache is touched
    k = cache.k[0].clone()
    with pytest.raises(ValueError, match="views"):
        net.extend(image, S.look_camera(64, 64, 100.0, (0.0, 0.0, 0.0)), cache)
    assert cache.tokens == 48 + 180 + 16 and int(cache.length) == cache.tokens
    assert torch.equal(cache.k[0].view(torch.int16), k.view(torch.int16))
