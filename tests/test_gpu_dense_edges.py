"""Edges of the gated feed-forward block and the 4-bit linear layers: the row
counts and widths at which another kernel or split is taken, long sums over
rows, broadcast rows that are not finite, two streams and two graphs at once,
and a run of the operators one after the other."""

import math

import pytest
import torch

import dense_oracle as O
from gaussian_splatting_differentiable_ewa_amd import tokens as T

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
DEV = "cuda"
NAMES = ("y", "gx", "gw_gate", "gw_up", "gw_down")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def weights(g, c, f, co, dtype):
    return ((rand(g, f, c) / math.sqrt(c)).to(dtype), (rand(g, f, c) / math.sqrt(c)).to(dtype),
            (rand(g, co, f) / math.sqrt(f)).to(dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows", [1, 4, 8, 9, 15, 16, 17])
@pytest.mark.parametrize("c,f,co", [(512, 520, 512), (520, 4096, 8), (8, 4104, 24), (1032, 16, 4104)])
def test_few_rows(dtype, rows, c, f, co):
    """Both sides of 8 and 16 rows, 4096 columns and sums of 512; y alone and what training keeps."""
    g = gen(rows + c)
    x, w = rand(g, rows, c, dtype=dtype), weights(g, c, f, co, dtype)
    gy = rand(g, rows, co, dtype=dtype)
    want = O.gated_ff(x, *w, "gelu", gy)
    y, h, kept = T.gated_ff_train(x, *w, "gelu")
    got = [y, *T.gated_ff_backward(gy, x, *w, h, kept, "gelu")]
    for name, p, (v, bound) in zip(NAMES, got, want):
        O.within(p, v, bound, name)
    assert torch.equal(T.gated_ff(x, *w, "gelu"), y)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,c,f,co", [(8161, 256, 520, 264), (20000, 40, 24, 16), (1111, 2056, 72, 8), (130, 8, 8200, 1032),
                                         (257, 4104, 264, 40), (63, 1032, 4104, 520)])
def test_long_sums(dtype, rows, c, f, co):
    """Sums over many rows or columns with few tiles: cut into splits of uneven length."""
    g = gen(rows + f)
    x, w = rand(g, rows, c, dtype=dtype), weights(g, c, f, co, dtype)
    gy = rand(g, rows, co, dtype=dtype)
    want = O.gated_ff(x, *w, "silu", gy)
    y, h, kept = T.gated_ff_train(x, *w)
    got = [y, *T.gated_ff_backward(gy, x, *w, h, kept)]
    for name, p, (v, bound) in zip(NAMES, got, want):
        O.within(p, v, bound, name)


@pytest.mark.parametrize("rows", [2, 50, 200])
def test_broadcast_rows_that_are_not_finite(rows):
    """One row of gy, or of x, for all, with an infinity: sums over rows of one sign stay infinite. The hidden layer and
    the gates are positive, and so is gy."""
    g = gen(rows)
    c, f, co = 64, 96, 40
    w = [t.abs() for t in weights(g, c, f, co, BF16)]
    x = rand(g, rows, c).abs().to(BF16)
    gy = rand(g, 1, co).abs().to(BF16).expand(rows, co).contiguous()
    y, h, kept = T.gated_ff_train(x, *w)
    gy[:, 3] = float("inf")
    wide = gy[:1].expand(rows, co)
    want = T.gated_ff_backward(gy, x, *w, h, kept)
    got = T.gated_ff_backward(wide, x, *w, h, kept)
    assert torch.equal(want[3][3], torch.full((f,), float("inf"), device=DEV, dtype=BF16))
    for p, r in zip(got, want):
        assert torch.equal(p.view(torch.int16), r.view(torch.int16))
    # x's row takes part in the projections' gradients; what was kept is of finite rows
    gy = rand(g, rows, co).abs().to(BF16)
    x1 = x[:1].clone()
    x1[0, 5] = float("inf")
    got = T.gated_ff_backward(gy, x1.expand(rows, c), *w, h, kept)
    want = T.gated_ff_backward(gy, x1.expand(rows, c).contiguous(), *w, h, kept)
    assert torch.equal(want[1][:, 5], torch.full((f,), float("inf"), device=DEV, dtype=BF16))
    for p, r in zip(got, want):
        assert torch.equal(p.view(torch.int16), r.view(torch.int16))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,c,n", [(1, 64, 1), (5, 32, 15), (8, 1056, 17), (16, 8192, 31), (17, 8192, 31), (16, 2080, 4097),
                                      (129, 4128, 129)])
def test_linear4_edges(dtype, rows, c, n):
    g = gen(rows + c)
    x, w = rand(g, rows, c, dtype=dtype), T.quantise4(rand(g, n, c) / math.sqrt(c))
    qx, qw = O.quantise4(x)[2], O.unpack4(*w, c)
    want = qx @ qw.T
    O.within(T.linear4(x, w), want, O.U[dtype] * want.abs() + (c + 16) * O.E * (qx.abs() @ qw.abs().T) + O.TINY[dtype], "y")


def test_linear4_weights_of_one_row_for_all():
    """Codes and scales with a row stride of zero: every column the same."""
    g = gen(1)
    w = T.quantise4(rand(g, 1, 96))
    for rows in (3, 70):
        x = rand(g, rows, 96, dtype=BF16)
        y = T.linear4(x, (w[0].expand(50, -1), w[1].expand(50, -1)))
        assert torch.equal(y, T.linear4(x, w).expand(rows, 50))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [1, 8, 32, 64])
def test_layer_norm_far_from_zero(dtype, c):
    """A constant row whose mean times 1 / sqrt(eps) passes fp32: x - mean is zero there, and the gradients are those
    of a constant row of ones, also in threads that hold columns past the row's. (Powers of two, of which the sum,
    2^127 at most, and the mean are exact; at other counts the mean's rounding squared passes fp32 in any form.)"""
    x = torch.ones(3, c, device=DEV)
    x[1] *= 2.0 ** 121
    x = x.to(dtype)
    gy = rand(gen(c), 1, c, dtype=dtype).expand(3, c).contiguous()
    w = 1 + rand(gen(c + 1), c) / 8
    y, stats = T.layer_norm(x, w)
    assert not y.any() and stats[0, 1] == 2.0 ** 121 and stats[1, 1] == stats[1, 0]
    gx, gw, gb = T.layer_norm_backward(gy, x, w, stats)
    assert torch.isfinite(gx).all() and torch.equal(gx[0], gx[1]) and torch.equal(gx[0], gx[2])
    assert not gw.any()
    O.within(gb, gy.double().sum(0), 3 * O.E * gy.double().abs().sum(0), "gb")


def block(x, ln, ff, four):
    """A layer as a model runs it: norm, feed-forward block and residual, and a head in 4 bits."""
    n, stats = T.layer_norm(x, *ln)
    y, h, kept = T.gated_ff_train(n, *ff, "gelu")
    out = T.linear4(x + y, four)
    gn, *gw = T.gated_ff_backward(y, n, *ff, h, kept, "gelu")
    gx, gl, gb = T.layer_norm_backward(gn, x, ln[0], stats)
    return [out, gx + y, gl, gb, *gw]


def block_inputs(seed, rows, c=136, f=264, n=72):
    g = gen(seed)
    c = (c + 31) // 32 * 32
    return (rand(g, rows, c, dtype=BF16), (1 + rand(g, c) / 8, rand(g, c) / 8), weights(g, c, f, c, BF16),
            T.quantise4(rand(g, n, c)))


def flat(inputs):
    x, ln, ff, four = inputs
    return [x, *ln, *ff, *four]


def test_a_run_of_them():
    """Through autograd and through the calls: the same bits, and near the 64-bit chain."""
    x, ln, ff, four = block_inputs(1, 90)
    y, gx, gl, gb, *gw = block(x, ln, ff, four)
    live = [t.clone().requires_grad_() for t in (x, *ln, *ff)]
    mid = T.GatedFF.apply(T.LayerNorm.apply(live[0], live[1], live[2]), *live[3:], "gelu")
    mid.backward(mid.detach())
    for p, t in zip((gl, gb, *gw), live[1:]):
        assert torch.equal(p, t.grad)
    n = O.layer_norm(x, *ln, 1e-5)
    a, _ = O.activation("gelu", n @ ff[0].double().T)
    want = (a * (n @ ff[1].double().T)) @ ff[2].double().T
    # 2^-8 of the magnitudes each: the norm through u, and through g (slope below 1.13), h and y
    size = ((a.abs() + n.abs() @ ff[0].double().abs().T) * (n.abs() @ ff[1].double().abs().T)) @ ff[2].double().abs().T
    assert ((mid.double() - want).abs() <= 5 * O.U[BF16] * size).all()


def test_two_streams_at_once():
    """The same calls on two streams with no wait between them."""
    sets = [block_inputs(s, rows) for s, rows in ((1, 300), (2, 1030), (3, 7))]
    want = [block(*i) for i in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, i in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(block(*i))
        torch.cuda.synchronize()
        for p, r in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(p, r))


def test_two_graphs_of_one_pool():
    """Captured steps of different sizes, replayed in turn with eager work between them, each on new inputs."""
    held = [block_inputs(0, 300), block_inputs(0, 17)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in held:
            block(*i)
    torch.cuda.current_stream().wait_stream(side)
    graphs, results = [torch.cuda.CUDAGraph() for _ in held], []
    for n, (graph, i) in enumerate(zip(graphs, held)):
        with torch.cuda.graph(graph, pool=graphs[0].pool() if n else None):
            results.append(block(*i))
    for seed in (1, 2, 3):
        for graph, i, out in zip(graphs, held, results):
            fresh = block_inputs(seed, i[0].shape[0])
            for t, u in zip(flat(i), flat(fresh)):
                t.copy_(u)
            graph.replay()
            got = [t.clone() for t in out]
            torch.cuda.synchronize()
            for p, r in zip(got, block(*fresh)):
                assert torch.equal(p, r), seed


def test_autograd_in_a_graph():
    """A training step through the autograd forms captured whole, gradients by autograd.grad; no eager graph of the
    same leaves is alive then. Every replay gives the eager bits."""
    def inputs(seed):
        x, ln, ff, _ = block_inputs(seed, 150)
        return [x, *ln, *ff, rand(gen(seed + 100), *x.shape, dtype=BF16)]

    def run(x, w, b, wg, wu, wd, gy):
        y = T.GatedFF.apply(T.LayerNorm.apply(x, w, b), wg, wu, wd, "silu")
        return [y.detach(), *torch.autograd.grad(y, (x, w, b, wg, wu, wd), gy)]

    held = inputs(0)
    for t in held[:-1]:
        t.requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = run(*held)
    for seed in (1, 2, 3):
        fresh = inputs(seed)
        with torch.no_grad():
            for t, u in zip(held, fresh):
                t.copy_(u)
        graph.replay()
        got = [t.clone() for t in results]
        torch.cuda.synchronize()
        for t in fresh[:-1]:
            t.requires_grad_()
        assert all(torch.equal(p, r) for p, r in zip(got, run(*fresh))), seed
