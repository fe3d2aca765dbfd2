"""The tiles and splits that the gated feed-forward block's cost model chooses
(csrc/gated_plan.h, compiled here by itself): the sizes that the GPU tests take
reach every form that it chooses for sizes over the whole range."""

import math
import os
import random
import subprocess

import pytest

import test_gpu_dense_edges
import test_gpu_gated_ff
import test_gpu_gated_ff_tiles
from gaussian_splatting_differentiable_ewa_amd import build

ASK = r"""
#include "gated_plan.h"
#include <cstdio>
int main()
{
    using namespace gs;
    long rows, c, f, co;
    while (std::scanf("%ld %ld %ld %ld", &rows, &c, &f, &co) == 4) {
        const Sizes z{rows, c, f, co};
        if (!sizes_ok(z) || !tiles_ok(z)) return 1;
        const int64_t m[3] = {rows, rows, rows}, n[3] = {f, co, f}, k[3] = {c, f, co};
        const int to[3] = {TO_GATED, TO_STORE, TO_GRAD};
        for (int i = 0; i < 3; ++i) {
            int shape;
            const Cut cut = cut_of(m[i], n[i], k[i], to[i], &shape);
            std::printf("%d %d ", shape, cut.splits);
        }
        const Back b = back_of(z);
        std::printf("%d %d %d %d\n", b.shape, b.c[0].splits, b.c[1].splits, b.c[2].splits);
    }
}
"""
FEW = 16  # rows that the forward pass takes without tiles


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    """Sizes -> the (product, tile, whether split) they take."""
    folder = tmp_path_factory.mktemp("plan")
    source, program = folder / "ask.cpp", folder / "ask"
    source.write_text(ASK)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-w", "-I", build.CSRC, "-o", str(program), str(source)],
                   check=True)

    def ask(sizes):
        text = "\n".join(" ".join(map(str, s)) for s in sizes)
        lines = subprocess.run([str(program)], input=text, text=True, capture_output=True, check=True).stdout.splitlines()
        assert len(lines) == len(sizes)
        found = set()
        for (rows, *_), line in zip(sizes, lines):
            h, hs, y, ys, g, gs, b, *bs = map(int, line.split())
            if rows > FEW:
                found |= {("h", h, hs > 1), ("y", y, ys > 1)}
            found |= {("gg and gu", g, gs > 1)} | {(name, b, s > 1) for name, s in zip(("gx", "gw_gate and gw_up", "gw_down"), bs)}
        return found

    return ask


def parameters(test, names):
    return next(list(m.args[1]) for m in test.pytestmark if m.name == "parametrize" and m.args[0] == names)


def test_every_form_is_tested(forms):
    rng = random.Random(7)

    def log(low, high):
        return round(math.exp(rng.uniform(math.log(low), math.log(high))))

    tested = [*test_gpu_gated_ff.SIZES, *test_gpu_gated_ff_tiles.SIZES,
              *parameters(test_gpu_dense_edges.test_long_sums, "rows,c,f,co")]
    chosen = forms([(log(1, 32640), 8 * log(1, 1024), 8 * log(1, 1024), 8 * log(1, 1024)) for _ in range(50000)])
    assert len(chosen) > 30 and not chosen - forms(tested), chosen - forms(tested)


@pytest.mark.parametrize("size,form", [((2048, 512, 1024, 512), ("h", 1, False)), ((3600, 256, 1024, 256), ("gg and gu", 1, False)),
                                       ((32640, 2048, 8192, 2048), ("gx", 2, False)), ((256, 256, 1024, 256), ("gx", 0, True))])
def test_forms_of_common_sizes(forms, size, form):
    assert form in forms([size])
