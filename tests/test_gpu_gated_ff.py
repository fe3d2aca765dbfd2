"""The gated feed-forward block on the GPU against its definition in 64 bits."""

import math

import pytest
import torch

import dense_oracle as O
from gaussian_splatting_differentiable_ewa_amd import _lib as L
from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
DEV = "cuda"
NAMES = ("y", "gx", "gw_gate", "gw_up", "gw_down")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def case(g, rows, c, f, co, dtype):
    """x, w_gate, w_up, w_down, gy."""
    return (rand(g, rows, c, dtype=dtype), (rand(g, f, c) / math.sqrt(c)).to(dtype), (rand(g, f, c) / math.sqrt(c)).to(dtype),
            (rand(g, co, f) / math.sqrt(f)).to(dtype), rand(g, rows, co, dtype=dtype))


# the least sizes; sizes off every tile and stage; rows from one on; few tiles cut along the sum, and tiles enough
SIZES = [(1, 8, 8, 8), (1, 520, 264, 72), (2, 64, 96, 40), (7, 2048, 1024, 256), (16, 72, 136, 80), (17, 256, 512, 256),
         (33, 40, 1032, 24), (64, 128, 128, 128), (65, 136, 200, 264), (300, 72, 520, 80), (257, 264, 1032, 136),
         (1000, 8, 16, 8), (2100, 72, 2056, 1032), (40, 2048, 2056, 2048), (8200, 1032, 1032, 1032)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,c,f,co", SIZES)
def test_both_ways(dtype, act, rows, c, f, co):
    g = gen(rows + c)
    x, wg, wu, wd, gy = case(g, rows, c, f, co, dtype)
    want = O.gated_ff(x, wg, wu, wd, act, gy)
    y, h, kept = T.gated_ff_train(x, wg, wu, wd, act)
    got = [y, *T.gated_ff_backward(gy, x, wg, wu, wd, h, kept, act)]
    for name, p, (w, bound) in zip(NAMES, got, want):
        assert p.dtype is dtype
        O.within(p, w, bound, name)
    assert torch.equal(T.gated_ff(x, wg, wu, wd, act), y)
    again = T.gated_ff_backward(gy, x, wg, wu, wd, h, kept, act)
    assert all(torch.equal(p, r) for p, r in zip(got[1:], again))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_against_differences(act):
    """The gradients through autograd along directions, against differences of
    the 64-bit form; fp16, so its roundings (2^-11 each, at most five on the way) are the bound."""
    g = gen(3)
    args = case(g, 24, 40, 48, 32, F16)
    gy = args[4]
    live = [t.clone().requires_grad_() for t in args[:4]]
    T.GatedFF.apply(*live, act).backward(gy)
    for n, t in enumerate(live):
        d = rand(g, *t.shape).double()

        def value(s):
            moved = [u.double() + (s * d if m == n else 0) for m, u in enumerate(args[:4])]
            a, _ = O.activation(act, moved[0] @ moved[1].T)
            return ((a * (moved[0] @ moved[2].T)) @ moved[3].T * gy.double()).sum()

        step = 1e-4
        slope = ((value(step) - value(-step)) / (2 * step)).item()
        assert abs((t.grad.double() * d).sum().item() - slope) <= 5 * O.U[F16] * (t.grad.double() * d).abs().sum().item() + 1e-6


def test_strides_and_alignment():
    """Views of packed matrices, and rows off 16 bytes (which are copied): the bits of contiguous tensors."""
    g = gen(4)
    rows, c, f = 70, 136, 200
    wide = rand(g, rows, 3 * c + 8, dtype=BF16)
    packed = (rand(g, 2 * f, c + 16) / math.sqrt(c)).to(BF16)
    down = (rand(g, c, f) / math.sqrt(f)).to(BF16)
    for first in (0, 8, 3):
        x, gy = wide[:, first: first + c], wide[:, first + c: first + 2 * c]
        wg, wu = packed[:f, first: first + c], packed[f:, first: first + c]
        wd = down.t().contiguous().t() if first == 3 else down
        y, h, kept = T.gated_ff_train(x, wg, wu, wd)
        grads = T.gated_ff_backward(gy, x, wg, wu, wd, h, kept)
        same = [t.contiguous() for t in (x, wg, wu, wd)]
        y2, h2, kept2 = T.gated_ff_train(*same)
        assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(kept, kept2)
        for p, r in zip(grads, T.gated_ff_backward(gy.contiguous(), *same, h2, kept2)):
            assert torch.equal(p, r)
    # one row for all (a row stride of zero), as x and as the gradient of a sum
    one = wide[:1, :c].expand(rows, c)
    y, h, kept = T.gated_ff_train(one, *same[1:])
    y2, h2, kept2 = T.gated_ff_train(one.contiguous(), *same[1:])
    assert torch.equal(y, y2)
    for p, r in zip(T.gated_ff_backward(one, one, *same[1:], h, kept),
                    T.gated_ff_backward(one.contiguous(), one.contiguous(), *same[1:], h2, kept2)):
        assert torch.equal(p, r)


@pytest.mark.parametrize("rows", [5, 200, 2304])
def test_what_is_not_finite_stays_in_its_row(rows):
    """NaN and infinity in a row of x reach y and gx of that row only, and a NaN row of gy gx of that row only;
    what lies behind the matrices in memory is not used."""
    g = gen(5)
    c, f, co = 72, 264, 136
    held = torch.full((rows + 1, c + 8), float("nan"), device=DEV, dtype=BF16)
    x0, wg, wu, wd, gy = case(g, rows, c, f, co, BF16)
    x = held[:rows, :c]
    x.copy_(x0)
    wg2 = torch.full((f + 1, c + 8), float("nan"), device=DEV, dtype=BF16)
    wg2[:f, :c] = wg
    clean = T.gated_ff_train(x0, wg, wu, wd)
    y, h, kept = T.gated_ff_train(x, wg2[:f, :c], wu, wd)
    assert torch.equal(y, clean[0])
    gx = T.gated_ff_backward(gy, x, wg2[:f, :c], wu, wd, h, kept)[0]
    x[1, 3], x[3, 5] = float("nan"), float("inf")
    y2, h2, kept2 = T.gated_ff_train(x, wg2[:f, :c], wu, wd)
    ok = torch.ones(rows, dtype=torch.bool, device=DEV)
    ok[[1, 3]] = False
    assert torch.equal(y2[ok], y[ok]) and torch.isnan(y2[1]).all() and not torch.isfinite(y2[3]).any()
    gy2 = gy.clone()
    gy2[4] = float("nan")
    gx2 = T.gated_ff_backward(gy2, x, wg2[:f, :c], wu, wd, h2, kept2)[0]
    ok[4] = False
    assert torch.equal(gx2[ok], gx[ok]) and torch.isnan(gx2[4]).all()


def test_no_rows_and_partial_gradients():
    g = gen(6)
    x, wg, wu, wd, gy = case(g, 0, 64, 96, 40, BF16)
    y, h, kept = T.gated_ff_train(x, wg, wu, wd)
    grads = T.gated_ff_backward(gy, x, wg, wu, wd, h, kept)
    assert y.shape == (0, 40) and grads[0].shape == (0, 64) and not any(t.any() for t in grads[1:])
    x, wg, wu, wd, gy = case(g, 50, 64, 96, 40, BF16)
    y, h, kept = T.gated_ff_train(x, wg, wu, wd)
    want = T.gated_ff_backward(gy, x, wg, wu, wd, h, kept)
    ws = torch.empty(L.gated_ff_bwd_workspace_bytes(50, 64, 96, 40), dtype=torch.uint8, device=DEV)
    for keep in ((0,), (1, 2), (3,)):
        got = [torch.full_like(t, 7.0) if n in keep else None for n, t in enumerate(want)]
        L.gs_gated_ff_bwd(gy, x, wg, wu, wd, h, kept, L.GS_SILU, *got, ws)
        assert all(torch.equal(got[n], want[n]) for n in keep)


def test_large_values():
    """The activations' ends: far negative gates close, far positive ones pass, nothing overflows on the way."""
    eye = torch.eye(8, device=DEV, dtype=BF16)
    x = torch.tensor([[-3e38, -1e4, -200.0, -90.0, 90.0, 200.0, 1e4, 1e18]], device=DEV).to(BF16)
    for act in ("silu", "gelu"):
        y, h, kept = T.gated_ff_train(x, eye, torch.full_like(eye, 0.0) + eye * 0.5, eye, act)
        want = torch.where(x < 0, 0.0, x.float() ** 2 / 2).to(BF16)
        assert torch.equal(y.abs(), want), act
        gx, *_ = T.gated_ff_backward(torch.ones_like(x), x, eye, eye * 0.5, eye, h, kept, act)
        assert torch.equal(gx.abs(), torch.where(x < 0, 0.0, x.float()).to(BF16)), act


def test_replays_equal_eager_calls():
    """Training steps captured in a graph, with new inputs and eager work between the replays; a second graph on
    the same memory pool does not disturb the first."""
    def inputs(seed):
        return list(case(gen(seed), 300, 136, 264, 72, BF16))

    def run(x, wg, wu, wd, gy):
        y, h, kept = T.gated_ff_train(x, wg, wu, wd, "gelu")
        return [y, h, kept, *T.gated_ff_backward(gy, x, wg, wu, wd, h, kept, "gelu"), T.gated_ff(x[:1], wg, wu, wd)]

    held = inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = run(*held)
    with torch.cuda.graph(other, pool=graph.pool()):
        more = run(*held)
    for seed in (0, 1, 2, 3):
        fresh = inputs(seed)
        for t, u in zip(held, fresh):
            t.copy_(u)
        graph.replay()
        got = [t.clone() for t in results]
        other.replay()
        got2 = [t.clone() for t in more]
        torch.cuda.synchronize()
        for p, q, r in zip(got, got2, run(*fresh)):
            assert torch.equal(p, r) and torch.equal(q, r), seed


def test_another_stream():
    """Calls go to the current stream, behind what it holds."""
    g = gen(7)
    x, wg, wu, wd, gy = case(g, 120, 64, 96, 64, F16)
    want = T.gated_ff(x, wg, wu, wd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        late = torch.zeros_like(x)
        for _ in range(50):
            late = late + 0.0 * x
        got = T.gated_ff(late + x, wg, wu, wd)
    side.synchronize()
    assert torch.equal(got, want)


def test_lost_gradients_are_refused():
    x, wg, wu, wd, _ = case(gen(8), 4, 16, 16, 16, BF16)
    wu.requires_grad_()
    with pytest.raises(ValueError):
        T.gated_ff(x, wg, wu, wd)
    with torch.no_grad():
        T.gated_ff(x, wg, wu, wd)
    y = T.GatedFF.apply(x, wg, wu, wd)
    first, = torch.autograd.grad(y.float().sum(), wu, create_graph=True)
    with pytest.raises(RuntimeError):
        first.float().sum().backward()
