// How the products of the gated feed-forward block (gated_ff.hip) are cut into
// tiles and splits: arithmetic of the host alone, without HIP, so that a program
// of its own can ask it too (tests/test_gated_plan.py).
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace gs {

// What becomes of a product's elements.
enum { TO_STORE = 0, TO_GATED = 1, TO_GRAD = 2 };

// Tiles of 64 x 64, 128 x 128 and 256 x 256.
enum { SMALL = 0, MID = 1, WIDE = 2 };
constexpr int64_t CUS = 256;

// How a product of m x n over k is cut into tiles of a shape and splits of the
// sum, and the time one block takes alone.
struct Cut {
    int32_t stages, splits, per_split;
    int64_t mt, nt, blocks;
    double us;
};

// Microseconds, by shape, as measured with 64 to 1024 blocks and k of 64 to 4096:
// a launch of blocks that do nothing else, a round of stages (one by each group)
// with few CUs at work and with all, and what an activation or its derivative
// adds at the end where the sum is not split. SLOTS blocks run at once.
static constexpr int64_t SIDE[3] = {64, 128, 256}, GROUPS[3] = {2, 2, 1}, SLOTS[3] = {2 * CUS, CUS, CUS};
static constexpr double LAUNCH[3] = {2.9, 2.9, 4.1}, ROUND[3] = {0.58, 0.89, 1.03}, ROUND_ALL[3] = {0.68, 1.49, 1.75};
static constexpr double ENDS[3][3] = {{0., 2.5, 3.}, {0., 4., 7.5}, {0., 7., 14.}};  // TO_STORE, TO_GATED, TO_GRAD

static Cut cut_as(int shape, int64_t m, int64_t wide, int64_t k, int segments, int64_t splits, int to)
{
    Cut c;
    c.mt = (m + SIDE[shape] - 1) / SIDE[shape];
    c.nt = (wide + SIDE[shape] - 1) / SIDE[shape];
    c.stages = (int32_t)((k + 63) / 64);
    const int64_t total = (int64_t)c.stages * segments;
    c.per_split = (int32_t)std::max<int64_t>(1, (total + splits - 1) / splits);
    c.splits = (int32_t)std::max<int64_t>(1, (total + c.per_split - 1) / c.per_split);
    c.blocks = c.mt * c.nt * c.splits;
    const double at_work = std::min(1.0, (double)c.blocks / CUS), round = ROUND[shape] + (ROUND_ALL[shape] - ROUND[shape]) * at_work;
    c.us = LAUNCH[shape] + round * (double)((c.per_split + GROUPS[shape] - 1) / GROUPS[shape]) + (c.splits > 1 ? 0. : ENDS[shape][to]);
    return c;
}

// Sums of splits are written, read and joined by another kernel: microseconds of
// its launch, with the gap before it (and half of what it takes on the host, which bounds
// small calls that are not in a graph), and of the sums.
constexpr double JOIN = 5.5;
static double sums_us(const Cut& c, int64_t m, int64_t wide) { return c.splits > 1 ? (double)(c.splits * m * wide) * 3e-6 : 0.; }

constexpr int64_t MOST_SPLITS = 32;

// The shape and splits that take the least time by the figures above.
static Cut cut_of(int64_t m, int64_t n, int64_t k, int to, int* shape)
{
    const int64_t wide = to == TO_GATED ? 2 * n : n;
    Cut best{};
    double least = 1e30;
    for (int s = SMALL; s <= WIDE; ++s)
        for (int64_t splits = 1; splits <= MOST_SPLITS; splits *= 2) {
            const Cut c = cut_as(s, m, wide, k, 1, splits, to);
            const double us = (double)((c.blocks + SLOTS[s] - 1) / SLOTS[s]) * c.us + sums_us(c, m, wide) + (c.splits > 1 ? JOIN : 0.);
            if (us < least) least = us, best = c, *shape = s;
            if (c.per_split <= 4) break;
        }
    return best;
}

static size_t part_bytes(const Cut& c, int64_t m, int64_t n, int to)
{
    return c.splits > 1 ? (size_t)c.splits * m * n * (to == TO_GATED ? 2 : 1) * 4 : 0;
}

struct Sizes {
    int64_t rows, c, f, co;
};

static bool sizes_ok(const Sizes& z)
{
    return z.rows >= 0 && z.rows <= (1 << 24) && z.c >= 8 && z.f >= 8 && z.co >= 8 && z.c <= (1 << 17) && z.f <= (1 << 17) &&
           z.co <= (1 << 17) && z.c % 8 == 0 && z.f % 8 == 0 && z.co % 8 == 0;
}

// The three products of the backward pass that need gg and gu, in one launch:
// gx, gWg and gWu over each other, gWd.
struct Back {
    int shape;
    Cut c[3];
    int64_t m[3], n[3];
    double us;
};

static Back back_of(const Sizes& z)
{
    const int64_t m[3] = {z.rows, 2 * z.f, z.co}, n[3] = {z.c, z.c, z.f}, k[3] = {z.f, z.rows, z.rows};
    Back best{};
    best.us = 1e30;
    for (int s = SMALL; s <= WIDE; ++s) {
        Back b{};
        b.shape = s;
        for (int i = 0; i < 3; ++i) b.m[i] = m[i], b.n[i] = n[i], b.c[i] = cut_as(s, m[i], n[i], k[i], i == 0 ? 2 : 1, 1, TO_STORE);
        // the longest blocks in splits, as long as that makes it shorter
        for (;;) {
            double sum = 0, longest = 0, joins = 0, sums = 0;
            int64_t blocks = 0;
            int which = 0;
            for (int i = 0; i < 3; ++i) {
                sum += b.c[i].us * (double)b.c[i].blocks;
                blocks += b.c[i].blocks;
                joins = std::max(joins, b.c[i].splits > 1 ? JOIN : 0.);  // one launch for all
                sums += sums_us(b.c[i], m[i], n[i]);
                if (b.c[i].us > longest) longest = b.c[i].us, which = i;
            }
            // whole rounds of the average block, or what a slot does on average and half of the longest block
            b.us = (blocks <= SLOTS[s] ? longest : sum / SLOTS[s] + longest / 2) + joins + sums;
            if (b.us < best.us) best = b;
            if (b.c[which].splits * 2 > MOST_SPLITS || b.c[which].per_split <= 4) break;
            b.c[which] = cut_as(s, m[which], n[which], k[which], which == 0 ? 2 : 1, b.c[which].splits * 2, TO_STORE);
        }
    }
    return best;
}

// Whether every product's workgroups, of 512 threads, are below 2^32
// threads.
static bool tiles_ok(const Sizes& z)
{
    int shape;
    const auto fits = [](int64_t blocks) { return blocks < (1 << 22); };
    const Back b = back_of(z);
    return fits(cut_of(z.rows, z.f, z.c, TO_GATED, &shape).blocks) && fits(cut_of(z.rows, z.co, z.f, TO_STORE, &shape).blocks) &&
           fits(cut_of(z.rows, z.f, z.co, TO_GRAD, &shape).blocks) && fits(b.c[0].blocks + b.c[1].blocks + b.c[2].blocks);
}

}  // namespace gs
